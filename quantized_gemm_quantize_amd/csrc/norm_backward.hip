// Gradients of the block norm (norm.hip), from those of its output o and of
// the new residual r' (d_new), given r' as stored:
//
//   s = 1 / rms(r'), h = s r':   d_r = d_new + s (d_o weight - h <d_o weight, h> / H)
//                                d_weight = sum_t d_o h
//   q = scale d_r, u the (normalized) block output:
//                                d_gate = q u (summed over rows for a vector)
//   p = q gate; without a post norm d_y = p; with one, z = 1 / rms(y), j = z y:
//                                d_post_weight = sum_t p j
//                                d_y = z (p post_weight - j <p post_weight, j> / H)
//
// Nothing is kept from the forward pass: both norms are made again from rows
// that the pass reads anyway. A workgroup runs through rows b, b + G, ... and
// keeps its threads' columns of the sums over rows in registers (fp32); at its
// end they go to partial[b], and a second kernel adds the G partials of each
// column in a fixed order, so repeated runs agree bit for bit.
// Bound by HBM: five (six with a gate row) reads and two (three) writes of
// T x H elements.
#include <algorithm>

#include "launch.hpp"
#include "norm.hpp"
#include "rows.hpp"

namespace block {
namespace {

using namespace rows;

template <Dtype D, int TPR, int C>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void backward_kernel(const Backward a) {
    typedef typename Element<D>::type E;
    constexpr int V = kPer<D>;
    constexpr int kThreads = TPR < 256 ? 256 : TPR;
    constexpr int kRows = kThreads / TPR;
    __shared__ float red[2][2][kThreads / kWave][3];  // by iteration parity and reduction
    __shared__ float columns[kRows > 1 ? (kRows - 1) * TPR * C * V : 1];
    w8a8::lds_poison(red);
    w8a8::lds_poison(columns);
    w8a8::lds_poison_done();
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int H = a.H;
    const bool has_y = a.y != nullptr, gate_rows = a.gate && a.ldg != 0, gate_vector = a.gate && a.ldg == 0;
    const float per = 1.0f / (float)H;

    float sw[C][V], sp[C][V], sg[C][V];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < V; ++e) sw[c][e] = sp[c][e] = sg[c][e] = 0.0f;

    int parity = 0;
    for (int64_t row = (int64_t)blockIdx.x * kRows + sub; row < a.T; row += (int64_t)gridDim.x * kRows, parity ^= 1) {
        uint4 ou[C], nu[C], ru[C], yu[C], gu[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = (c * TPR + t) * V;
            ou[c] = nu[c] = ru[c] = yu[c] = gu[c] = make_uint4(0, 0, 0, 0);
            if (k < H) {
                ou[c] = load_chunk<D, true>(static_cast<const E *>(a.d_out) + row * a.ldo, k, H);
                ru[c] = load_chunk<D, true>(static_cast<const E *>(a.residual) + row * a.ldr, k, H);
                if (has_y) yu[c] = load_chunk<D, true>(static_cast<const E *>(a.y) + row * a.ldy, k, H);
                if (a.d_new) nu[c] = load_chunk<D, true>(static_cast<const E *>(a.d_new) + row * a.ldn, k, H);
                if (gate_rows) gu[c] = load_chunk<D, true>(static_cast<const E *>(a.gate) + row * a.ldg, k, H);
            }
        }
        // <r', r'>, <y, y>, <d_o weight, r'>
        float sums[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = (c * TPR + t) * V;
            if (k >= H) continue;
            float o[V], r[V], y[V], w[V];
            widen_chunk<D>(ou[c], o);
            widen_chunk<D>(ru[c], r);
            widen_chunk<D>(yu[c], y);
            load_vector<D>(a.weight, k, H, 1.0f, w);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                sums[0] = __builtin_fmaf(r[e], r[e], sums[0]);
                sums[1] = __builtin_fmaf(y[e], y[e], sums[1]);
                sums[2] = __builtin_fmaf(o[e] * w[e], r[e], sums[2]);
            }
        }
        row_sums<TPR>(sums, red[parity][0]);
        const float s = 1.0f / __builtin_sqrtf(sums[0] * per + a.eps);
        const float z = 1.0f / __builtin_sqrtf(sums[1] * per + a.eps);
        const float along = s * s * sums[2] * per;   // d_r = d_new + s (d_o weight - r' along)
        float p[C][V];   // the gradient of the (normalized) block output, times post_weight
        float dot[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = (c * TPR + t) * V;
            if (k >= H) continue;
            float o[V], r[V], w[V], n[V], d[V];
            widen_chunk<D>(ou[c], o);
            widen_chunk<D>(ru[c], r);
            widen_chunk<D>(nu[c], n);
            load_vector<D>(a.weight, k, H, 1.0f, w);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                d[e] = __builtin_fmaf(s, o[e] * w[e] - r[e] * along, n[e]);
                sw[c][e] = __builtin_fmaf(o[e], r[e] * s, sw[c][e]);
            }
            store_chunk<D>(static_cast<E *>(a.d_residual) + row * H, k, H, narrow_chunk<D>(d));
            if (!has_y) continue;
            float y[V], pw[V], f[V];
            widen_chunk<D>(yu[c], y);
            load_vector<D>(a.post ? a.post_weight : nullptr, k, H, 1.0f, pw);
            if (gate_rows) widen_chunk<D>(gu[c], f);
            else load_vector<D>(gate_vector ? static_cast<const float *>(a.gate) : nullptr, k, H, 1.0f, f);
            const float unit = a.post ? z : 1.0f;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float q = a.scale * d[e], j = y[e] * unit, g = q * f[e];
                d[e] = q * (j * pw[e]);                        // the gate's gradient
                sg[c][e] += d[e];
                sp[c][e] = __builtin_fmaf(g, j, sp[c][e]);
                p[c][e] = g * pw[e];
                dot[0] = __builtin_fmaf(p[c][e], y[e], dot[0]);
            }
            if (gate_rows && a.d_gate)
                store_chunk<D>(static_cast<E *>(a.d_gate) + row * H, k, H, narrow_chunk<D>(d));
        }
        if (!has_y) continue;
        if (a.post) row_sums<TPR>(dot, reinterpret_cast<float (*)[1]>(red[parity][1]));
        const float back = z * z * dot[0] * per;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = (c * TPR + t) * V;
            if (k >= H) continue;
            if (a.post) {
                float y[V];
                widen_chunk<D>(yu[c], y);
#pragma unroll
                for (int e = 0; e < V; ++e) p[c][e] = z * (p[c][e] - y[e] * back);
            }
            store_chunk<D>(static_cast<E *>(a.d_y) + row * H, k, H, narrow_chunk<D>(p[c]));
        }
    }

    // the rows of one workgroup, then its partial sums
    int at = 0;
    auto give = [&](float (&s)[C][V]) {
        if constexpr (kRows > 1) {
            __syncthreads();
            if (sub > 0)
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int e = 0; e < V; ++e) columns[((sub - 1) * C * V + c * V + e) * TPR + t] = s[c][e];
            __syncthreads();
            if (sub > 0) {
                ++at;
                return;
            }
#pragma unroll
            for (int o = 0; o < kRows - 1; ++o)
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int e = 0; e < V; ++e) s[c][e] += columns[(o * C * V + c * V + e) * TPR + t];
        }
        float *to = a.partial + ((int64_t)at * gridDim.x + blockIdx.x) * H;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = (c * TPR + t) * V;
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (k + e < H) to[k + e] = s[c][e];
        }
        ++at;
    };
    if (a.d_weight) give(sw);
    if (a.d_post_weight) give(sp);
    if (a.d_gate && gate_vector) give(sg);
}

// out[h] = sum over G partials of column h, in a fixed order: SLICES slices of
// the partials, each in order, then the slices.
struct Sums {
    float *out[3];
};
constexpr int kColumns = 64, kSlices = 16;

__global__ __launch_bounds__(kColumns *kSlices) void sum_partials(const float *__restrict__ partial, int G, int H,
                                                                  Sums to) {
    __shared__ float red[kSlices][kColumns];
    w8a8::lds_poison(red);
    w8a8::lds_poison_done();
    const int c = threadIdx.x % kColumns, slice = threadIdx.x / kColumns;
    const int h = blockIdx.x * kColumns + c;
    const float *from = partial + (int64_t)blockIdx.y * G * H + h;
    float s = 0.0f;
    if (h < H)
        for (int g = slice; g < G; g += kSlices) s += from[(int64_t)g * H];
    red[slice][c] = s;
    __syncthreads();
    if (slice || h >= H) return;
#pragma unroll
    for (int i = 1; i < kSlices; ++i) s += red[i][c];
    to.out[blockIdx.y][h] = s;
}

int workgroups(int64_t T, int rows) {
    return (int)std::min<int64_t>((T + rows - 1) / rows, kBackwardWorkgroups);
}

template <Dtype D, int TPR, int C>
hipError_t launch(const Backward &a, hipStream_t stream) {
    constexpr int kThreads = TPR < 256 ? 256 : TPR;
    const int G = workgroups(a.T, kThreads / TPR);
    if (G) {
        backward_kernel<D, TPR, C><<<dim3((unsigned)G), dim3(kThreads), 0, stream>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    Sums to{};
    int n = 0;
    if (a.d_weight) to.out[n++] = a.d_weight;
    if (a.d_post_weight) to.out[n++] = a.d_post_weight;
    if (a.d_gate && a.ldg == 0) to.out[n++] = static_cast<float *>(a.d_gate);
    if (!n) return hipSuccess;
    sum_partials<<<dim3((unsigned)((a.H + kColumns - 1) / kColumns), (unsigned)n), dim3(kColumns * kSlices), 0,
                   stream>>>(a.partial, G, a.H, to);
    return hipGetLastError();
}

template <Dtype D>
hipError_t launch_row(const Backward &a, hipStream_t stream) {
    constexpr int V = kPer<D>;
    const int chunks = (a.H + V - 1) / V;
    if (chunks <= 64) return launch<D, 64, 1>(a, stream);
    if (chunks <= 128) return launch<D, 64, 2>(a, stream);
    if (chunks <= 256) return launch<D, 256, 1>(a, stream);
    if (chunks <= 512) return launch<D, 256, 2>(a, stream);
    if (chunks <= 1024) return launch<D, 256, 4>(a, stream);
    if constexpr (D == kF32) {
        if (chunks > 2048) return launch<D, 1024, 4>(a, stream);
    }
    return launch<D, 1024, 2>(a, stream);
}

}  // namespace

int64_t backward_workspace(int64_t T, int64_t H) {
    return 4 * 3 * H * std::min<int64_t>(T, kBackwardWorkgroups);
}

hipError_t launch_backward(const Backward &a, int dtype, hipStream_t stream) {
    switch (dtype) {
        case kBf16: return launch_row<kBf16>(a, stream);
        case kF16: return launch_row<kF16>(a, stream);
        default: return launch_row<kF32>(a, stream);
    }
}

}  // namespace block
