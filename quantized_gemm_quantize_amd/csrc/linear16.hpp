// Arguments of the 16-bit products (linear16.hip) and their epilogue.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace linear16 {

// out[m][n] = round(act(acc + bias[n]) + residual[m][n]), pre[m][n] = round(acc + bias[n])
struct Epilogue {
    const float *bias;      // null: none
    const void *residual;   // null: none
    int64_t ldr;
    void *pre;              // null: not wanted
    void *out;
    int act;
};

// One operand of a product over k: element (row, k) at p[row * ld + k], or, k-major, at
// p[k * ld + row].
struct Operand {
    const void *p;
    int64_t ld;
    bool k_major;
};

// The tiles of a product, how many of them (the first ones in the tile order) one workgroup computes
// whole, and how many workgroups share each other one along k.
enum Form { k64x64, k128x128deep, k128x128, k256x128, k256x256, k64x64deep, kForms };
struct Plan {
    Form form;
    int whole, splits;
    int64_t workspace;   // bytes of partial sums
};

hipError_t launch_tiled(const Operand &a, const Operand &b, int64_t M, int64_t N, int64_t K, bool f16, const Plan &plan,
                        float *partial, const Epilogue &ep, hipStream_t stream);

// The int8 product (bf16 outputs, whole tiles of the wavefronts that take stages of their own), K a
// multiple of 16; its sums are scaled by rows and channels before the epilogue.
hipError_t launch_int8(const int8_t *xq, const float *x_scale, int64_t M, const int8_t *wq, const float *w_scale, int64_t N,
                       int64_t K, const Epilogue &ep, hipStream_t stream);

// d_x and d_w in one launch: plain products of one form, b k-major, a of w too. The workgroups of one
// come first.
struct Product {
    Operand a, b;
    int64_t M, N, K;
    void *out;
};
struct PairPlan {
    Plan x, w;
    bool w_first;
};

hipError_t launch_pair(const Product &x, const Product &w, bool f16, const PairPlan &plan, float *partial,
                       hipStream_t stream);

// What a call launches, and the workspace that it needs.
struct ForwardPlan {
    bool rows;              // launch_rows
    Plan tiles;
    int64_t workspace() const { return rows ? 0 : tiles.workspace; }
};
struct BackwardPlan {
    PairPlan both;          // where both gradients are wanted
    Plan x, w;              // of one alone
    int64_t workspace;
};
ForwardPlan plan_forward(int64_t M, int64_t N, int64_t K);
BackwardPlan plan_backward(int64_t M, int64_t N, int64_t K);

// The product of up to kMaxRows rows, in one launch without a workspace.
constexpr int kMaxRows = 64;
// Up to so many rows a call may leave its workspace out: launch_rows stands for any other plan.
constexpr int kNoWorkspaceRows = 16;
hipError_t launch_rows(const void *x, int64_t ldx, int M, const void *w, int N, int K, bool f16, const Epilogue &ep,
                       hipStream_t stream);

}  // namespace linear16
