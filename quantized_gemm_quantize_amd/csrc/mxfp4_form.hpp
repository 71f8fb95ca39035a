// The kernel that a product takes (chosen in mxfp4_gemm.hip, launched by the kernels' files).
#pragma once

#include <stdint.h>

namespace mxfp4 {

// A workgroup's part of the outputs: rows x channels, by so many wavefronts of the
// weight-streaming kernel (stream) or the LDS-tiled one.
struct Form {
    bool stream;
    int rows, channels, waves;
};

// Rows of a product: S of them, or S in E groups.
struct Rows {
    int64_t S, E;
    bool grouped;
};

Form product_form(const Rows &r, int N, int K, int epilogue, int64_t cus);

// Whether the launch is within a grid's threads.
bool product_fits(const Rows &r, int N, int K, int epilogue);

}  // namespace mxfp4
