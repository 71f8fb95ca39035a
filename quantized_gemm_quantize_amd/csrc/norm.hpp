// Arguments of the block norm kernels (norm.hip, norm_backward.hip).
#pragma once

#include <stdint.h>

namespace block {

// What a row becomes for the next block.
enum Out { kSame = 0, kInt8 = 1, kMxfp4 = 2 };

struct Forward {
    const void *residual, *y, *gate;   // rows; y null: no block output
    int64_t ldr, ldy, ldg;             // gate with ldg 0: an fp32 vector
    const float *post_weight, *weight; // null: ones
    int post;
    float scale, eps;
    int64_t T;
    int H;
    void *new_residual;
    void *out;                         // rows of the dtype, int8 codes or MXFP4 codes
    void *out_scale;                   // fp32 per row, or MXFP4 scale codes
};

struct Backward {
    const void *d_out, *d_new, *residual, *y, *gate;  // d_new null: zeros; residual: the new one
    int64_t ldo, ldn, ldr, ldy, ldg;
    const float *post_weight, *weight;
    int post;
    float scale, eps;
    int64_t T;
    int H;
    void *d_residual, *d_y, *d_gate;                  // d_gate null: not wanted
    float *d_weight, *d_post_weight;                  // null: not wanted
    float *partial;                                   // [workgroups][sums][H]
};

}  // namespace block
