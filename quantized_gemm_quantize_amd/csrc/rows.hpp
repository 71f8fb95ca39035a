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

// The elements [k, min(k + kPer, width)) of a row as one chunk, zeros behind its end. STREAM: read
// only this once. WHOLE: rows of whole chunks. Other rows are loaded in two parts: a load that every
// thread makes without a branch, of the row's last kPer elements where the chunk ends behind it, and,
// when the chunk is used, the shift of those into their places. (Element loads in a branch wait there,
// which ends what is in flight: 2864 x 1189 backward 52 us, without 31. Rows of whole chunks have no use for
// it: 8192 x 4096 backward 103, with it 128.) Rows shorter than a chunk are loaded by elements.
template <Dtype D, bool WHOLE, bool STREAM>
__device__ __forceinline__ uint4 load_chunk(const typename Element<D>::type *row, int k, int width) {
    typedef typename std::conditional<D == kF32, loose16w, loose16>::type V;
    if (WHOLE ? k < width : width >= kPer<D>) {
        const V *p = reinterpret_cast<const V *>(row + (WHOLE ? k : min(k, width - kPer<D>)));
        w8a8::v4i v;
        if constexpr (STREAM) v = __builtin_nontemporal_load(p);
        else v = *p;
        return __builtin_bit_cast(uint4, v);
    }
    uint32_t w[4] = {0, 0, 0, 0};
    if constexpr (!WHOLE)
#pragma unroll
        for (int e = 0; e < kPer<D>; ++e)
            if (k + e < width) {
                if constexpr (D == kF32) w[e] = __float_as_uint(row[k + e]);
                else w[e / 2] |= (uint32_t)row[k + e] << (16 * (e & 1));
            }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <Dtype D, bool WHOLE>
__device__ __forceinline__ uint4 settle(uint4 u, int k, int width) {
    if constexpr (WHOLE) return u;
    const int behind = k + kPer<D> - width;   // elements
    if (behind <= 0 || width < kPer<D>) return u;
    if (behind >= kPer<D>) return make_uint4(0, 0, 0, 0);
    const int bits = behind * 8 * kSize<D>;
    uint64_t lo = u.x | (uint64_t)u.y << 32, hi = u.z | (uint64_t)u.w << 32;
    if (bits >= 64) {
        lo = hi >> (bits - 64);
        hi = 0;
    } else {
        lo = lo >> bits | hi << (64 - bits);
        hi >>= bits;
    }
    return make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32));
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

template <Dtype D, bool WHOLE>
__device__ __forceinline__ void store_chunk(typename Element<D>::type *row, int k, int width, uint4 u) {
    typedef typename std::conditional<D == kF32, loose16w, loose16>::type V;
    if (WHOLE ? k < width : k + kPer<D> <= width) {
        *reinterpret_cast<V *>(row + k) = __builtin_bit_cast(w8a8::v4i, u);
        return;
    }
    if constexpr (WHOLE) return;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < kPer<D>; ++e)
        if (k + e < width) {
            if constexpr (D == kF32) row[k + e] = __uint_as_float(w[e]);
            else row[k + e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
        }
}

// kPer floats of a vector [width] (parameters, kept in fp32): `none` for a null vector, and any finite
// numbers behind the end.
template <Dtype D, bool WHOLE>
__device__ __forceinline__ void load_vector(const float *p, int k, int width, float none, float (&v)[kPer<D>]) {
#pragma unroll
    for (int e = 0; e < kPer<D>; ++e) v[e] = none;
    if (!p || k >= width) return;
#pragma unroll
    for (int q = 0; q < kPer<D>; q += 4) {
        const uint4 u = settle<kF32, WHOLE>(load_chunk<kF32, WHOLE, false>(p, k + q, width), k + q, width);
        widen_chunk<kF32>(u, reinterpret_cast<float (&)[4]>(v[q]));
    }
}

// f(v, v of the lane whose number differs in bit OFF), of a commutative f; for OFF of 4 and 8 the
// lanes that differ in lower bits hold the same v already, and a mirrored row stands for the exchange.
// Exchanges inside the vector registers take a few cycles each, those through the LDS crossbar 100.
template <int OFF, class F>
__device__ __forceinline__ uint32_t across(uint32_t v, F f) {
    if constexpr (OFF >= 16) {
        const auto p = OFF == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                                 : __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return f((uint32_t)p[0], (uint32_t)p[1]);
    } else {
        // quad_perm [1,0,3,2] and [2,3,0,1], row_half_mirror, row_mirror
        constexpr int kControl = OFF == 1 ? 0xB1 : OFF == 2 ? 0x4E : OFF == 4 ? 0x141 : 0x140;
        return f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, kControl, 0xF, 0xF, true));
    }
}

template <int TPR, class F>
__device__ __forceinline__ uint32_t across_row(uint32_t v, F f) {
    static_assert(TPR == 16 || TPR % kWave == 0, "whole rows of lanes");
    v = across<8>(across<4>(across<2>(across<1>(v, f), f), f), f);
    if constexpr (TPR >= kWave) v = across<32>(across<16>(v, f), f);
    return v;
}

// Sums of N values over the TPR threads of a row: 16 lanes, a wavefront, or all of a workgroup's TPR
// threads (then every thread calls it, and `red` is not used again before another barrier). The order
// is fixed: repeated runs agree bit for bit.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&s)[N], float (*red)[N]) {
    const auto add = [](uint32_t x, uint32_t y) {
        return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
    };
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = __uint_as_float(across_row<TPR>(__float_as_uint(s[i]), add));
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

// Hides a chunk's value from the compiler: what was computed from it before is computed again
// from the 4 registers instead of being kept in up to 8.
__device__ __forceinline__ void forget(uint4 &u) { asm volatile("" : "+v"(u.x), "+v"(u.y), "+v"(u.z), "+v"(u.w)); }

}  // namespace rows
