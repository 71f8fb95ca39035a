// Quantization of rows to MXFP4 (device side).
//
// Per block of 32 elements along the row: code = exponent of the largest
// magnitude - 2 (scale_code), then every element is x / 2^(code - 127)
// rounded half to even to e2m1 and saturated at 6. Dividing by a power of two
// is exact, so gfx950's scaled conversions (v_cvt_scalef32_pk_fp4_*) compute
// exactly that, bf16 / binary16 / binary32 and subnormals alike.
//
// 32 lanes take one row's 256 elements (16 bytes of 16-bit input per lane, two
// such loads of 32-bit input), four lanes share a block (two lane swaps for its
// largest magnitude), and each 32-lane half writes 128 bytes of codes and the 8
// scale bytes of its step.
#pragma once

#include "mxfp4.hpp"

namespace mxfp4 {

typedef unsigned short v2u __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(v2u, a),
                                                                  __builtin_bit_cast(v2u, b)));
}

// 8 consecutive elements as loaded, their largest magnitude, and their codes.
template <Dtype D>
struct Eight {
    uint4 u[D == kF32 ? 2 : 1];

    __device__ __forceinline__ void load(const void *p) {
        u[0] = w8a8::load16_stream(p);
        if constexpr (D == kF32) u[1] = w8a8::load16_stream(static_cast<const char *>(p) + 16);
    }
    __device__ __forceinline__ void clear() {
        u[0] = make_uint4(0, 0, 0, 0);
        if constexpr (D == kF32) u[1] = u[0];
    }
    // bit pattern of the largest magnitude (of each half word for 16-bit types)
    __device__ __forceinline__ uint32_t top() const {
        if constexpr (D == kF32) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m = max(m, max(u[i].x & 0x7FFFFFFFu, u[i].y & 0x7FFFFFFFu));
                m = max(m, max(u[i].z & 0x7FFFFFFFu, u[i].w & 0x7FFFFFFFu));
            }
            return m;
        } else {
            const uint32_t k = 0x7FFF7FFFu;
            return max_u16x2(max_u16x2(u[0].x & k, u[0].y & k), max_u16x2(u[0].z & k, u[0].w & k));
        }
    }
    __device__ __forceinline__ static uint32_t merge(uint32_t a, uint32_t b) {
        if constexpr (D == kF32) return max(a, b);
        else return max_u16x2(a, b);
    }
    __device__ __forceinline__ static float top_value(uint32_t m) {
        if constexpr (D == kF32) return __uint_as_float(m);
        else {
            const uint32_t h = max(m & 0xFFFFu, m >> 16);
            if constexpr (D == kBf16) return __uint_as_float(h << 16);
            else return (float)__builtin_bit_cast(_Float16, (unsigned short)h);
        }
    }
    __device__ __forceinline__ uint32_t codes(float scale) const {
        uint32_t r = 0;
        if constexpr (D == kF32) {
            const float *f = reinterpret_cast<const float *>(u);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[0], f[1], scale, 0);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[2], f[3], scale, 1);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[4], f[5], scale, 2);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[6], f[7], scale, 3);
        } else if constexpr (D == kBf16) {
            using w8a8::v2bf;
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(v2bf, u[0].x), scale, 0);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(v2bf, u[0].y), scale, 1);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(v2bf, u[0].z), scale, 2);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(v2bf, u[0].w), scale, 3);
        } else {
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(v2h, u[0].x), scale, 0);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(v2h, u[0].y), scale, 1);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(v2h, u[0].z), scale, 2);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(v2h, u[0].w), scale, 3);
        }
        return r;
    }
};

// Steps of the matrix (256 elements; step u is step u % KB of row u / KB) of
// workgroup `block` of THREADS threads: THREADS / 32 * U consecutive ones, each
// 32-lane half every (THREADS / 32)-th of them, all loads first.
template <Dtype D, int U, int THREADS>
__device__ __forceinline__ void quantize_steps(int64_t block, const char *__restrict__ x, int64_t ldx,
                                               int64_t M, int K, int KB, uint8_t *__restrict__ codes,
                                               uint8_t *__restrict__ scales) {
    constexpr int kHalves = THREADS / 32;
    constexpr int kSize = D == kF32 ? 4 : 2;
    const int half = threadIdx.x >> 5, i = threadIdx.x & 31;
    const int64_t first = block * (kHalves * U);
    const int64_t row0 = first / KB;
    const int step0 = (int)(first - row0 * KB);
    Eight<D> v[U];
    int64_t row[U];
    int step[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const uint32_t s = (uint32_t)(step0 + half + j * kHalves);
        const uint32_t r = s / (uint32_t)KB;
        row[j] = row0 + r;
        step[j] = (int)(s - r * KB);
        const int k = step[j] * kStep + 8 * i;
        v[j].clear();
        if (row[j] < M && k < K) v[j].load(x + (row[j] * ldx + k) * kSize);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
        if (row[j] >= M) continue;  // uniform per half
        uint32_t m = v[j].top();
        m = Eight<D>::merge(m, (uint32_t)__shfl_xor((int)m, 1, kWave));
        m = Eight<D>::merge(m, (uint32_t)__shfl_xor((int)m, 2, kWave));
        const uint32_t code = scale_code(Eight<D>::top_value(m));
        const int k = step[j] * kStep + 8 * i;
        if (k < K) {
            const uint32_t c = code == 255 ? 0u : v[j].codes(scale_value(code));
            *reinterpret_cast<uint32_t *>(codes + row[j] * (K / 2) + k / 2) = c;
        }
        // lanes past K hold zeros and write the padding's code 0
        if (i % 4 == 0) scales[((int64_t)step[j] * M + row[j]) * 8 + i / 4] = (uint8_t)code;
    }
}

}  // namespace mxfp4
