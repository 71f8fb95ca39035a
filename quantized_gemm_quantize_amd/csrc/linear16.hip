// 16-bit products with bias, activation and residual, and their gradients.
//
//   forward   pre = x w^T + bias, out = act(pre) + residual
//   backward  d_pre = d_out act'(pre), d_bias = sum_m d_out act'(pre),
//             d_x = d_pre w, d_w = d_pre^T x
//
// One kernel for the three products: 64 x 64 tiles, 16 steps of k in LDS as
// binary32, 4 x 4 outputs per thread.
#include <algorithm>

#include "activation.hpp"
#include "launch.hpp"
#include "linear16.hpp"
#include "rows.hpp"

namespace linear16 {
namespace {

using namespace rows;

constexpr int kTile = 64, kDepth = 16;

template <Dtype D>
__global__ __launch_bounds__(256) void product_kernel(Operand a, Operand b, int64_t M, int64_t N, int64_t K, Epilogue ep) {
    __shared__ float ta[kDepth][kTile + 1], tb[kDepth][kTile + 1];
    w8a8::lds_poison(ta);
    w8a8::lds_poison(tb);
    w8a8::lds_poison_done();
    const int64_t tiles_n = (N + kTile - 1) / kTile;
    const int64_t m0 = blockIdx.x / tiles_n * kTile, n0 = blockIdx.x % tiles_n * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    auto load = [&](const Operand &o, int64_t r0, int64_t rows, int64_t k0, float (&to)[kDepth][kTile + 1]) {
        for (int i = threadIdx.x; i < kDepth * kTile; i += 256) {
            const int r = o.k_major ? i % kTile : i / kDepth, k = o.k_major ? i / kTile : i % kDepth;
            float v = 0.0f;
            if (r0 + r < rows && k0 + k < K)
                v = widen<D>(static_cast<const uint16_t *>(o.p)[o.k_major ? (k0 + k) * o.ld + r0 + r : (r0 + r) * o.ld + k0 + k]);
            to[k][r] = v;
        }
    };
    for (int64_t k0 = 0; k0 < K; k0 += kDepth) {
        load(a, m0, M, k0, ta);
        load(b, n0, N, k0, tb);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kDepth; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_fmaf(ta[k][ty * 4 + i], tb[k][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + tx + 16 * j;
            v[j] = acc[i][j];
            if (m < M && n < N) {
                if (ep.bias) v[j] += ep.bias[n];
                if (ep.pre) static_cast<uint16_t *>(ep.pre)[m * N + n] = narrow<D>(v[j]);
            }
        }
        act::activate(ep.act, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + tx + 16 * j;
            if (m >= M || n >= N) continue;
            if (ep.residual) v[j] += widen<D>(static_cast<const uint16_t *>(ep.residual)[m * ep.ldr + n]);
            static_cast<uint16_t *>(ep.out)[m * N + n] = narrow<D>(v[j]);
        }
    }
}

template <int A, Dtype D>
__device__ __forceinline__ float d_value(float d, float p) { return d * act::slope<A>(p); }

// d_pre and the column sums of d_out act'(pre): a workgroup takes every G-th
// block of rows of 64 columns and leaves one partial sum per column.
template <Dtype D>
__global__ __launch_bounds__(256) void slope_kernel(const uint16_t *d_out, int64_t ldd, const uint16_t *pre, int64_t M,
                                                    int64_t N, int a, uint16_t *d_pre, float *partial) {
    __shared__ float red[4][64];
    w8a8::lds_poison(red);
    w8a8::lds_poison_done();
    const int c = threadIdx.x % 64, s = threadIdx.x / 64;
    const int64_t n = (int64_t)blockIdx.x * 64 + c;
    float sum = 0.0f;
    if (n < N)
        for (int64_t m = blockIdx.y * 4 + s; m < M; m += gridDim.y * 4) {
            float d = widen<D>(d_out[m * ldd + n]);
            if (a != act::kNone) {
                const float p = widen<D>(pre[m * N + n]);
                d *= a == act::kRelu ? act::slope<act::kRelu>(p) : a == act::kGelu ? act::slope<act::kGelu>(p)
                   : a == act::kGeluTanh ? act::slope<act::kGeluTanh>(p) : act::slope<act::kSilu>(p);
                d_pre[m * N + n] = narrow<D>(d);
            }
            sum += d;
        }
    if (!partial) return;
    red[s][c] = sum;
    __syncthreads();
    if (s || n >= N) return;
    for (int i = 1; i < 4; ++i) sum += red[i][c];
    partial[blockIdx.y * N + n] = sum;
}

__global__ __launch_bounds__(256) void sum_kernel(const float *partial, int G, int64_t N, float *out) {
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n >= N) return;
    float s = 0.0f;
    for (int g = 0; g < G; ++g) s += partial[g * N + n];
    out[n] = s;
}

int sum_groups(int64_t M) { return (int)std::min<int64_t>(64, (M + 3) / 4); }

hipError_t product(Operand a, Operand b, int64_t M, int64_t N, int64_t K, bool f16, const Epilogue &ep, hipStream_t stream) {
    const dim3 grid((unsigned)(((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile)));
    if (f16) product_kernel<kF16><<<grid, 256, 0, stream>>>(a, b, M, N, K, ep);
    else product_kernel<kBf16><<<grid, 256, 0, stream>>>(a, b, M, N, K, ep);
    return hipGetLastError();
}

}  // namespace

int64_t forward_workspace(int64_t, int64_t, int64_t) { return 0; }

int64_t backward_workspace(int64_t M, int64_t N, int64_t) { return 4 * N * sum_groups(M); }

hipError_t launch_forward(const void *x, int64_t ldx, int64_t M, const void *w, int64_t N, int64_t K, bool f16,
                          const Epilogue &ep, void *, hipStream_t stream) {
    return product({x, ldx, false}, {w, K, false}, M, N, K, f16, ep, stream);
}

hipError_t launch_backward(const void *d_out, int64_t ldd, const void *x, int64_t ldx, const void *w, const void *pre,
                           int64_t M, int64_t N, int64_t K, bool f16, int a, void *d_pre, void *d_x, void *d_w,
                           float *d_bias, void *workspace, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (a != act::kNone || d_bias) {
        const int G = sum_groups(M);
        const dim3 grid((unsigned)((N + 63) / 64), (unsigned)G);
        float *partial = d_bias ? static_cast<float *>(workspace) : nullptr;
        const uint16_t *d = static_cast<const uint16_t *>(d_out), *p = static_cast<const uint16_t *>(pre);
        uint16_t *to = static_cast<uint16_t *>(d_pre);
        if (G) {
            if (f16) slope_kernel<kF16><<<grid, 256, 0, stream>>>(d, ldd, p, M, N, a, to, partial);
            else slope_kernel<kBf16><<<grid, 256, 0, stream>>>(d, ldd, p, M, N, a, to, partial);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        if (d_bias) {
            sum_kernel<<<dim3((unsigned)((N + 255) / 256)), 256, 0, stream>>>(partial, G, N, d_bias);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
    }
    if (a == act::kNone) d_pre = const_cast<void *>(d_out);
    const int64_t ld = a == act::kNone ? ldd : N;
    if (d_x && M && (e = product({d_pre, ld, false}, {w, K, true}, M, K, N, f16, Epilogue{nullptr, nullptr, 0, nullptr, d_x, 0}, stream)) != hipSuccess)
        return e;
    if (d_w) return product({d_pre, ld, true}, {x, ldx, true}, N, K, M, f16, Epilogue{nullptr, nullptr, 0, nullptr, d_w, 0}, stream);
    return hipSuccess;
}

}  // namespace linear16
