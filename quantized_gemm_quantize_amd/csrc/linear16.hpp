// Arguments of the 16-bit products (linear16.hip) and their epilogue.
#pragma once

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

}  // namespace linear16
