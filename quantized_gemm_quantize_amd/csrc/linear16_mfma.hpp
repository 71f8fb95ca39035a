// Matrix instructions and LDS layout that the 16-bit products share (device side).
#pragma once

#include "common.hpp"

namespace linear16 {

using w8a8::kWave;
using w8a8::v4i;

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(1))) void global_void;

// 16 x 16 outputs, 32 k: lane l holds row l % 16 of each operand, k 8 (l / 16) ... + 7. Output:
// lane l, element r: row 4 (l / 16) + r of a, row l % 16 of b. On random operands this form runs
// 1990 TFLOP/s where the 32 x 32 x 16 one runs 1730: the card is at its power limit, and this one
// moves its accumulators half as often.
template <bool F16>
__device__ __forceinline__ v4f mfma(v4i a, v4i b, v4f c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// Rows of 64 k lie in LDS as 8 chunks of 16 bytes, chunk c of row r at slot c ^ swz(r). A 16-byte
// LDS read serves lanes 0-3, 12-15 and 20-27 (of each 32) in one pass and the others in the next
// (measured): of a fragment those are rows 0-3 and 12-15 of one chunk and rows 4-11 of its
// neighbour, which then lie in 16 distinct 16-byte banks, as do the others.
__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }

}  // namespace linear16
