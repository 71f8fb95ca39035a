// Rows of bf16, binary16 or binary32 in chunks of 16 bytes, as the row kernels
// hold them: loads and stores that need the element's alignment only (the
// hardware takes any address; rows of odd widths start anywhere), and sums over
// the threads of a row.
#pragma once

#include <type_traits>

#include "mxfp4.hpp"

namespace rows {

using mxfp4::kBf16;
using mxfp4::kF16;
using mxfp4::kF32;
using mxfp4::Dtype;
using w8a8::kWave;

template <Dtype D> struct Element { typedef uint16_t type; };
template <> struct Element<kF32> { typedef float type; };

template <Dtype D> constexpr int kSize = D == kF32 ? 4 : 2;
template <Dtype D> constexpr int kPer = 16 / kSize<D>;   // elements of a chunk

// 16 bytes at an address that is aligned to an element
typedef w8a8::v4i loose16 __attribute__((aligned(2)));
typedef w8a8::v4i loose16w __attribute__((aligned(4)));

template <Dtype D>
__device__ __forceinline__ float widen(typename Element<D>::type e) {
    if constexpr (D == kF32) return e;
    else if constexpr (D == kBf16) return __uint_as_float((uint32_t)e << 16);
    else return (float)__builtin_bit_cast(_Float16, e);
}

template <Dtype D>
__device__ __forceinline__ typename Element<D>::type narrow(float f) {
    if constexpr (D == kF32) return f;
    else if constexpr (D == kBf16) return __builtin_bit_cast(uint16_t, (__bf16)f);
    else return __builtin_bit_cast(uint16_t, (_Float16)f);
}

// The elements [k, min(k + kPer, width)) of a row as one chunk, zeros behind
// its end. STREAM: read only this once.
template <Dtype D, bool STREAM>
__device__ __forceinline__ uint4 load_chunk(const typename Element<D>::type *row, int k, int width) {
    typedef typename std::conditional<D == kF32, loose16w, loose16>::type V;
    if (k + kPer<D> <= width) {
        const V *p = reinterpret_cast<const V *>(row + k);
        w8a8::v4i v;
        if constexpr (STREAM) v = __builtin_nontemporal_load(p);
        else v = *p;
        return __builtin_bit_cast(uint4, v);
    }
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < kPer<D>; ++e)
        if (k + e < width) {
            if constexpr (D == kF32) w[e] = __float_as_uint(row[k + e]);
            else w[e / 2] |= (uint32_t)row[k + e] << (16 * (e & 1));
        }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <Dtype D>
__device__ __forceinline__ void widen_chunk(uint4 u, float (&v)[kPer<D>]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < kPer<D>; ++e) {
        if constexpr (D == kF32) v[e] = __uint_as_float(w[e]);
        else v[e] = widen<D>((uint16_t)(w[e / 2] >> (16 * (e & 1))));
    }
}

template <Dtype D>
__device__ __forceinline__ uint4 narrow_chunk(const float (&v)[kPer<D>]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (D == kF32) w[e] = __float_as_uint(v[e]);
        else if constexpr (D == kBf16) w[e] = w8a8::pack_bf16x2(v[2 * e], v[2 * e + 1]);
        else {
            const mxfp4::v2h h = {(_Float16)v[2 * e], (_Float16)v[2 * e + 1]};
            w[e] = __builtin_bit_cast(uint32_t, h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <Dtype D>
__device__ __forceinline__ void store_chunk(typename Element<D>::type *row, int k, int width, uint4 u) {
    typedef typename std::conditional<D == kF32, loose16w, loose16>::type V;
    if (k + kPer<D> <= width) {
        *reinterpret_cast<V *>(row + k) = __builtin_bit_cast(w8a8::v4i, u);
        return;
    }
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < kPer<D>; ++e)
        if (k + e < width) {
            if constexpr (D == kF32) row[k + e] = __uint_as_float(w[e]);
            else row[k + e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
        }
}

// kPer floats of a vector [width] (parameters, kept in fp32), `none` for a null
// vector and behind the end.
template <Dtype D>
__device__ __forceinline__ void load_vector(const float *p, int k, int width, float none,
                                            float (&v)[kPer<D>]) {
#pragma unroll
    for (int e = 0; e < kPer<D>; ++e) v[e] = none;
    if (!p) return;
    if (k + kPer<D> <= width) {
#pragma unroll
        for (int q = 0; q < kPer<D> / 4; ++q) {
            const float4 f = *reinterpret_cast<const float4 *>(p + k + 4 * q);
            v[4 * q] = f.x; v[4 * q + 1] = f.y; v[4 * q + 2] = f.z; v[4 * q + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < kPer<D>; ++e)
            if (k + e < width) v[e] = p[k + e];
    }
}

// Sums of N values over the TPR threads of a row (64, or all of a workgroup's
// TPR threads: then every thread calls it, and `red` is not used again before
// another barrier). The order is fixed: repeated runs agree bit for bit.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&s)[N], float (*red)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) s[i] += __shfl_xor(s[i], off, kWave);
    if constexpr (TPR > kWave) {
        const int wave = threadIdx.x / kWave;
        if (threadIdx.x % kWave == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) red[wave][i] = s[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            s[i] = red[0][i];
#pragma unroll
            for (int w = 1; w < TPR / kWave; ++w) s[i] += red[w][i];
        }
    }
}

}  // namespace rows
