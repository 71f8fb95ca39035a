// Activations of the product epilogues and their derivatives (device side), in
// binary32.
//
//   relu      max(v, 0)                    v > 0
//   gelu      v P(v)                       P(v) + v p(v)
//   gelu_tanh v s(z(v))                    s + v s (1 - s) z'(v)
//   silu      v s(v)                       s + v s (1 - s)
//
// with P and p the normal distribution and its density, s(x) = 1 / (1 + e^-x)
// and z(v) = 2 sqrt(2 / pi) (v + 0.044715 v^3) (gelu's tanh form: (1 + tanh y) / 2
// = s(2 y)). s and 1 - s come from e^-|x| <= 1, so neither cancels nor
// overflows; the exponential is taken 2^32 times too large and scaled back last,
// because the hardware's 2^x flushes subnormal results, which would lose
// silu(v) below v = -87 (its value is 87 times larger than e^v).
// P(-a) = e^(-a^2/2) t Q(t), t = 1 / (1 + 0.28 a): a minimax fit of the
// scaled complementary error function over a >= 0 (relative error 1.7e-7), so
// gelu keeps its precision in the lower tail, where (1 + erf) / 2 has none left.
// Infinite v give the limits (0 on the left, v on the right; slopes 0 and 1), NaN gives NaN (relu's
// slope 0): factors that meet an exponential of 0 are bounded first.
#pragma once

#include "common.hpp"

namespace act {

enum Activation { kNone = 0, kRelu = 1, kGelu = 2, kGeluTanh = 3, kSilu = 4 };

constexpr float kLog2e = 1.44269504088896341f;

// e^x for x <= 0: `big` is 2^32 times it, `e` itself (subnormals kept).
struct Decay {
    float big, e;
    __device__ __forceinline__ explicit Decay(float x) {
        big = __builtin_amdgcn_exp2f(__builtin_fmaf(x, kLog2e, 32.0f));
        e = big * 0x1p-32f;
    }
};

// s(x) * u (u of x's sign, or positive) and, with `other`, 1 - s(x).
__device__ __forceinline__ float sigmoid_times(float x, float u, float &other) {
    const Decay d(-__builtin_fabsf(x));
    const float r = __builtin_amdgcn_rcpf(1.0f + d.e);
    other = x < 0 ? r : d.e * r;
    return x < 0 ? fmaxf(u, -0x1p64f) * d.big * r * 0x1p-32f : u * r;
}

// z(v) of the tanh form; an infinite cube keeps its sign.
__device__ __forceinline__ float tanh_argument(float v) {
    constexpr float c = 1.59576912160573071f;  // 2 sqrt(2 / pi)
    return c * __builtin_fmaf(0.044715f * v * v, v, v);
}

// P(-a) for a >= 0, 2^32 times too large.
__device__ __forceinline__ float lower_tail_big(float a, const Decay &d) {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.28f, a, 1.0f));
    float q = 0.024761965f;
    q = __builtin_fmaf(q, t, -0.0937581010f);
    q = __builtin_fmaf(q, t, 0.0926925140f);
    q = __builtin_fmaf(q, t, -0.00667161348f);
    q = __builtin_fmaf(q, t, 0.0728802850f);
    q = __builtin_fmaf(q, t, 0.0836029219f);
    q = __builtin_fmaf(q, t, 0.103088515f);
    q = __builtin_fmaf(q, t, 0.111699568f);
    q = __builtin_fmaf(q, t, 0.111703862f);
    return d.big * (t * q);
}

template <int A>
__device__ __forceinline__ float value(float v) {
    float unused;
    if constexpr (A == kRelu) return v < 0 ? 0.0f : v;
    if constexpr (A == kSilu) return sigmoid_times(v, v, unused);
    if constexpr (A == kGeluTanh) return sigmoid_times(tanh_argument(v), v, unused);
    if constexpr (A == kGelu) {
        const float a = fminf(__builtin_fabsf(v), 64.0f);   // the tail ends before
        const float tail = a * lower_tail_big(a, Decay(-0.5f * a * a)) * 0x1p-32f;
        return v < 0 ? -tail : v - tail;
    }
    return v;
}

template <int A>
__device__ __forceinline__ float slope(float v) {
    if constexpr (A == kRelu) return v > 0 ? 1.0f : 0.0f;
    if constexpr (A == kSilu) {
        float other;
        const float s = sigmoid_times(v, 1.0f, other);
        return s == 0.0f || other == 0.0f ? s : __builtin_fmaf(v * s, other, s);
    }
    if constexpr (A == kGeluTanh) {
        constexpr float c = 1.59576912160573071f, c3 = 3 * 0.044715f * c;
        float other;
        const float s = sigmoid_times(tanh_argument(v), 1.0f, other);
        // where one side of s is 0 the other is the slope (v^2 may be infinite)
        return s == 0.0f || other == 0.0f ? s
                                          : __builtin_fmaf(v * s * other, __builtin_fmaf(c3 * v, v, c), s);
    }
    if constexpr (A == kGelu) {
        constexpr float density = 0.398942280401432678f;  // 1 / sqrt(2 pi)
        const float a = __builtin_fabsf(v);
        const Decay d(-0.5f * a * a);
        const float tail = lower_tail_big(a, d) * 0x1p-32f, p = v < 0 ? tail : 1.0f - tail;
        return d.e == 0.0f ? p : __builtin_fmaf(v * density, d.e, p);
    }
    return 1.0f;
}

// The same for N values, the activation chosen at run time (uniform).
template <int A, int N>
__device__ __forceinline__ void values(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = value<A>(v[i]);
}

template <int N>
__device__ __forceinline__ void activate(int a, float (&v)[N]) {
    switch (a) {
        case kRelu: values<kRelu>(v); break;
        case kGelu: values<kGelu>(v); break;
        case kGeluTanh: values<kGeluTanh>(v); break;
        case kSilu: values<kSilu>(v); break;
        default: break;
    }
}

}  // namespace act
