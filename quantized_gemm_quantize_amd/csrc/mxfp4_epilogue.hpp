// What the MXFP4 products do with a wavefront's accumulators.
#pragma once

#include "mxfp4.hpp"

namespace mxfp4 {

// Where a product's outputs go: out [S, N] of Dtype, or (SwiGLU) the hidden
// activations [S, N/2] in MXFP4.
struct Output {
    void *out;
    uint8_t *codes, *scales;
};

enum Epilogue { kOutBf16 = kBf16, kOutF16 = kF16, kOutF32 = kF32, kSwiglu = 3 };

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, v2h{(_Float16)lo, (_Float16)hi});
}

// SwiGLU of two neighbouring 32-channel tiles (64 channels: gate and up rows
// alternate, so 32 hidden units, one MXFP4 block) and the quantization of the
// block. A lane holds units 16 jj + 4 g + 2 half + 0..1 of row m (jj: tile);
// the two halves join their largest magnitudes and swap codes so that each
// writes 8 consecutive bytes. The activations are never rounded in between.
struct Hidden {
    uint2 codes;    // bytes 8 half .. + 7 of the block's 16
    uint32_t code;  // its scale
};

__device__ __forceinline__ Hidden quantize_swiglu(const v16f &lo, const v16f &hi, int half) {
    float h[2][8];
    uint32_t top = 0;
#pragma unroll
    for (int jj = 0; jj < 2; ++jj)
#pragma unroll
        for (int u = 0; u < 8; u += 4) {
            const v16f &a = jj ? hi : lo;
            const v4f v = swiglu4(v4f{a[2 * u], a[2 * u + 2], a[2 * u + 4], a[2 * u + 6]},
                                  v4f{a[2 * u + 1], a[2 * u + 3], a[2 * u + 5], a[2 * u + 7]});
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[jj][u + i] = v[i];
                top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
            }
        }
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, kWave));
    const uint32_t code = scale_code(__uint_as_float(top));
    const float scale = scale_value(code);
    uint32_t c[2];
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
        uint32_t r = 0;
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, h[jj][0], h[jj][1], scale, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, h[jj][2], h[jj][3], scale, 1);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, h[jj][4], h[jj][5], scale, 2);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, h[jj][6], h[jj][7], scale, 3);
        c[jj] = code == 255 ? 0u : r;
    }
    // byte 8 jj + 2 g + half of the block's 16; this lane writes bytes 8 half .. +7
    const uint32_t keep = half ? c[1] : c[0], give = half ? c[0] : c[1];
    const uint32_t take = (uint32_t)__shfl_xor((int)give, 32, kWave);
    const uint32_t even = half ? take : keep, odd = half ? keep : take;
    return Hidden{make_uint2(__builtin_amdgcn_perm(odd, even, 0x05010400u),
                             __builtin_amdgcn_perm(odd, even, 0x07030602u)),
                  code};
}

// The block of hidden units of channels n0 .. n0 + 63 of row m; with the last
// block of a row, the zeros that pad its scales.
__device__ __forceinline__ void store_hidden(const Hidden &h, const Output &o, int64_t m, bool live,
                                             int n0, int half, int N, int S) {
    const int F = N / 2, f0 = n0 / 2;  // this block's first hidden unit
    if (!live || f0 >= F) return;
    *reinterpret_cast<uint2 *>(o.codes + m * (F / 2) + f0 / 2 + 8 * half) = h.codes;
    if (half == 0) {
        uint8_t *s = o.scales + ((int64_t)(f0 / kStep) * S + m) * 8;
        const int b = (f0 / 32) % 8;
        s[b] = (uint8_t)h.code;
        if (f0 + 32 == F)
            for (int i = b + 1; i < 8; ++i) s[i] = 0;
    }
}

}  // namespace mxfp4
