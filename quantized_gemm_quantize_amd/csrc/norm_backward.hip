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
// Bound by HBM: four reads (d_o, d_new, r', y; five with a gate row) and two (three) writes of
// T x H elements. Measured, both kernels: 8192 x 4096 bf16 with post norm and gate rows 91 us (5.9 TB/s), in
// 32 bits 189 (5.7), 16448 x 1280 bf16 with a gate vector 64 us (3.9), 4096 x 8192 105 (3.8), 1000 x 16384 110 (1.8:
// its rows are read three times, and 250 partial sums of three vectors joined); a single row 5 us.
#include <algorithm>

#include "launch.hpp"
#include "norm.hpp"
#include "rows.hpp"

namespace block {
namespace {

using namespace rows;

// Most workgroups that leave partial sums.
int most_partials(int64_t H) { return H <= 2048 ? 768 : H <= 4096 ? 512 : 256; }

constexpr int kOneWorkgroup = 4;   // rows

// A row's operands as loaded.
template <Dtype D, bool WHOLE, int TPR, int C>
struct Row {
    uint4 o[C], n[C], r[C], y[C], g[C];

    // chunk c of this thread
    template <bool STREAM>
    __device__ __forceinline__ void load(const Backward &a, int64_t row, int t, int c, bool gate_rows) {
        typedef typename Element<D>::type E;
        const int k = (c * TPR + t) * kPer<D>;
        n[c] = y[c] = g[c] = make_uint4(0, 0, 0, 0);
        o[c] = load_chunk<D, WHOLE, STREAM>(static_cast<const E *>(a.d_out) + row * a.ldo, k, a.H);
        r[c] = load_chunk<D, WHOLE, STREAM>(static_cast<const E *>(a.residual) + row * a.ldr, k, a.H);
        if (a.y) y[c] = load_chunk<D, WHOLE, STREAM>(static_cast<const E *>(a.y) + row * a.ldy, k, a.H);
        if (a.d_new) n[c] = load_chunk<D, WHOLE, STREAM>(static_cast<const E *>(a.d_new) + row * a.ldn, k, a.H);
        if (gate_rows) g[c] = load_chunk<D, WHOLE, STREAM>(static_cast<const E *>(a.gate) + row * a.ldg, k, a.H);
    }
    __device__ __forceinline__ void settled(int t, int c, int H) {
        const int k = (c * TPR + t) * kPer<D>;
        o[c] = settle<D, WHOLE>(o[c], k, H);
        n[c] = settle<D, WHOLE>(n[c], k, H);
        r[c] = settle<D, WHOLE>(r[c], k, H);
        y[c] = settle<D, WHOLE>(y[c], k, H);
        g[c] = settle<D, WHOLE>(g[c], k, H);
    }
};

// POST: a post norm; GATE: none, a vector or rows. (Their sums and vectors would cost registers where
// they are not there: 101 of 16-bit rows without either, 140 with both.)
enum Gate { kNone, kVector, kRowsOf };

template <Dtype D, bool WHOLE, int TPR, int C, bool POST, Gate GATE>
__global__ __launch_bounds__(TPR <= kWave ? 256 : TPR) void backward_kernel(const Backward a) {
    typedef typename Element<D>::type E;
    constexpr int V = kPer<D>;
    constexpr int kThreads = TPR <= kWave ? 256 : TPR;
    constexpr int kRows = kThreads / TPR;
    // a row's loads are on their way while the one before is computed, where registers allow it
    // (4096 x 5120: 126 -> 103 us); of one chunk per thread the vectors stay in registers, too
    constexpr bool kKept = C == 1, kAhead = kKept || (WHOLE && TPR < 1024);
    // Rows of several chunks to each of 1024 threads do not fit in registers beside their sums; they
    // are read again where they are used (1000 x 16384: held and spilled 253 us, read again 175).
    constexpr bool kAgain = C > 1 && TPR == 1024;
    __shared__ float red[2][2][kThreads / kWave][3];  // by iteration parity and reduction
    __shared__ float columns[kRows > 1 ? (kRows - 1) * TPR * C * V : 1];
    w8a8::lds_poison(red);
    w8a8::lds_poison(columns);
    w8a8::lds_poison_done();
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int H = a.H;
    const bool has_y = a.y != nullptr;
    const float *const gate = static_cast<const float *>(a.gate);   // GATE == kVector
    const float per = 1.0f / (float)H;

    float sw[C][V] = {}, sp[C][V] = {}, sg[C][V] = {};   // of weight, post weight, a gate vector
    float kept[kKept ? 3 : 1][V];   // weight, post weight, gate
    if constexpr (kKept) {
        load_vector<D, WHOLE>(a.weight, t * V, H, 1.0f, kept[0]);
        if constexpr (POST) load_vector<D, WHOLE>(a.post_weight, t * V, H, 1.0f, kept[1]);
        if constexpr (GATE == kVector) load_vector<D, WHOLE>(gate, t * V, H, 1.0f, kept[2]);
    }
    auto vector = [&](int which, const float *p, int k, float (&v)[V]) {
        if constexpr (kKept) {
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = kept[which][e];
        } else {
            load_vector<D, WHOLE>(p, k, H, 1.0f, v);
        }
    };

    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + sub;
    Row<D, WHOLE, TPR, C> u, ahead;
    auto load = [&](Row<D, WHOLE, TPR, C> &into, int64_t row) {
#pragma unroll
        for (int c = 0; c < C; ++c) into.template load<true>(a, row, t, c, GATE == kRowsOf);
    };
    auto again = [&](int64_t row, int c) {
        if constexpr (kAgain) {
            asm volatile("" ::: "memory");   // one chunk at a time
            u.template load<false>(a, row, t, c, GATE == kRowsOf);
            u.settled(t, c, H);
        }
    };
    if (!kAgain && row < a.T) load(ahead, row);
    for (int parity = 0; row < a.T; row += step, parity ^= 1) {
        if constexpr (!kAgain) {
            u = ahead;
#pragma unroll
            for (int c = 0; c < C; ++c) u.settled(t, c, H);
            if (kAhead && row + step < a.T) load(ahead, row + step);
        }
        // <r', r'>, <y, y>, <d_o weight, r'>
        float sums[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = (c * TPR + t) * V;
            if (k >= H) continue;
            again(row, c);
            float o[V], r[V], y[V], w[V];
            widen_chunk<D>(u.o[c], o);
            widen_chunk<D>(u.r[c], r);
            widen_chunk<D>(u.y[c], y);
            vector(0, a.weight, k, w);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                sums[0] = __builtin_fmaf(r[e], r[e], sums[0]);
                if constexpr (POST) sums[1] = __builtin_fmaf(y[e], y[e], sums[1]);
                sums[2] = __builtin_fmaf(o[e] * w[e], r[e], sums[2]);
            }
            forget(u.o[c]);
            forget(u.r[c]);
            forget(u.y[c]);
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
            again(row, c);
            float o[V], r[V], w[V], n[V], d[V];
            widen_chunk<D>(u.o[c], o);
            widen_chunk<D>(u.r[c], r);
            widen_chunk<D>(u.n[c], n);
            vector(0, a.weight, k, w);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                d[e] = __builtin_fmaf(s, o[e] * w[e] - r[e] * along, n[e]);
                sw[c][e] = __builtin_fmaf(o[e], r[e] * s, sw[c][e]);
            }
            store_chunk<D, WHOLE>(static_cast<E *>(a.d_residual) + row * H, k, H, narrow_chunk<D>(d));
            if (!has_y) continue;
            float y[V], pw[V], f[V];
            widen_chunk<D>(u.y[c], y);
            if constexpr (POST) vector(1, a.post_weight, k, pw);
            if constexpr (GATE == kRowsOf) widen_chunk<D>(u.g[c], f);
            if constexpr (GATE == kVector) vector(2, gate, k, f);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float q = a.scale * d[e], j = POST ? y[e] * z : y[e], g = GATE != kNone ? q * f[e] : q;
                if constexpr (GATE != kNone) d[e] = q * (POST ? j * pw[e] : j);   // the gate's gradient
                if constexpr (GATE == kVector) sg[c][e] += d[e];
                p[c][e] = g;
                if constexpr (POST) {
                    sp[c][e] = __builtin_fmaf(g, j, sp[c][e]);
                    p[c][e] = g * pw[e];
                    dot[0] = __builtin_fmaf(p[c][e], y[e], dot[0]);
                }
            }
            if (GATE == kRowsOf && a.d_gate)
                store_chunk<D, WHOLE>(static_cast<E *>(a.d_gate) + row * H, k, H, narrow_chunk<D>(d));
        }
        if (has_y) {
            if constexpr (POST) row_sums<TPR>(dot, reinterpret_cast<float (*)[1]>(red[parity][1]));
            const float back = z * z * dot[0] * per;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = (c * TPR + t) * V;
                if (k >= H) continue;
                if constexpr (POST) {
                    float y[V];
                    forget(u.y[c]);
                    if constexpr (kAgain) {
                        asm volatile("" ::: "memory");
                        u.y[c] = load_chunk<D, WHOLE, false>(static_cast<const E *>(a.y) + row * a.ldy, k, H);
                        u.y[c] = settle<D, WHOLE>(u.y[c], k, H);
                    }
                    widen_chunk<D>(u.y[c], y);
#pragma unroll
                    for (int e = 0; e < V; ++e) p[c][e] = z * (p[c][e] - y[e] * back);
                }
                store_chunk<D, WHOLE>(static_cast<E *>(a.d_y) + row * H, k, H, narrow_chunk<D>(p[c]));
            }
        }
        if (!kAhead && !kAgain && row + step < a.T) load(ahead, row + step);
    }

    // the rows of one workgroup, then its partial sums (the results, where it is alone)
    int at = 0;
    auto give = [&](float (&s)[C][V], float *alone) {
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
        float *to = gridDim.x == 1 ? alone : a.partial + ((int64_t)at * gridDim.x + blockIdx.x) * H;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = (c * TPR + t) * V;
#pragma unroll
            for (int q = 0; q < V; q += 4)
                store_chunk<kF32, WHOLE>(to, k + q, H, narrow_chunk<kF32>(reinterpret_cast<float (&)[4]>(s[c][q])));
        }
        ++at;
    };
    if (a.d_weight) give(sw, a.d_weight);
    if (POST && a.d_post_weight) give(sp, a.d_post_weight);
    if (GATE == kVector && a.d_gate) give(sg, static_cast<float *>(a.d_gate));
}

// out[h] = sum over G partials of column h, in a fixed order: slices of the partials, each in
// order, then the slices.
struct Sums {
    float *out[3];
};
constexpr int kColumns = 32, kSlices = 32;

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
#pragma unroll 8
        for (int g = slice; g < G; g += kSlices) s += from[(int64_t)g * H];
    red[slice][c] = s;
    __syncthreads();
    if (slice || h >= H) return;
#pragma unroll
    for (int i = 1; i < kSlices; ++i) s += red[i][c];
    to.out[blockIdx.y][h] = s;
}

// Workgroups: as many as are resident at once (of 12 wavefronts per CU that their registers allow, 16
// of 32-bit rows), each with the same number of rows (1000 x 16384, 512 workgroups with a row or two
// each 175 us, 250 with four each 109; 615 x 2692 33 -> 20); a few rows go to one, which needs no
// second launch (one row of 4096 8 -> 5 us).
template <Dtype D>
int workgroups(int64_t T, int64_t H, int threads, int rows) {
    if (T <= std::max(rows, kOneWorkgroup)) return T > 0;
    const int64_t resident = 256 * std::max(1, (D == kF32 ? 16 : 12) * kWave / threads);
    const int64_t most = std::min<int64_t>(resident, most_partials(H));
    const int64_t steps = (T + rows * most - 1) / (rows * most);
    return (int)((T + rows * steps - 1) / (rows * steps));
}

template <Dtype D, bool WHOLE, int TPR, int C, bool POST>
void launch_gate(const Backward &a, int G, hipStream_t stream) {
    constexpr int kThreads = TPR <= kWave ? 256 : TPR;
    const dim3 grid((unsigned)G), block(kThreads);
    if (!a.gate) backward_kernel<D, WHOLE, TPR, C, POST, kNone><<<grid, block, 0, stream>>>(a);
    else if (a.ldg == 0) backward_kernel<D, WHOLE, TPR, C, POST, kVector><<<grid, block, 0, stream>>>(a);
    else backward_kernel<D, WHOLE, TPR, C, POST, kRowsOf><<<grid, block, 0, stream>>>(a);
}

template <Dtype D, int TPR, int C>
hipError_t launch(const Backward &a, hipStream_t stream) {
    constexpr int kThreads = TPR <= kWave ? 256 : TPR;
    const int G = workgroups<D>(a.T, a.H, kThreads, kThreads / TPR);
    if (G) {
        if (a.H % kPer<D> == 0) a.post ? launch_gate<D, true, TPR, C, true>(a, G, stream) : launch_gate<D, true, TPR, C, false>(a, G, stream);
        else a.post ? launch_gate<D, false, TPR, C, true>(a, G, stream) : launch_gate<D, false, TPR, C, false>(a, G, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    Sums to{};
    int n = 0;
    if (a.d_weight) to.out[n++] = a.d_weight;
    if (a.d_post_weight) to.out[n++] = a.d_post_weight;
    if (a.d_gate && a.ldg == 0) to.out[n++] = static_cast<float *>(a.d_gate);
    if (!n || G == 1) return hipSuccess;
    sum_partials<<<dim3((unsigned)((a.H + kColumns - 1) / kColumns), (unsigned)n), dim3(kColumns * kSlices), 0,
                   stream>>>(a.partial, G, a.H, to);
    return hipGetLastError();
}

template <Dtype D>
hipError_t launch_row(const Backward &a, hipStream_t stream) {
    constexpr int V = kPer<D>;
    const int chunks = (a.H + V - 1) / V;
    if (chunks <= 16) return launch<D, 16, 1>(a, stream);
    if (chunks <= 64) return launch<D, 64, 1>(a, stream);
    if (chunks <= 256) return launch<D, 256, 1>(a, stream);
    if (chunks <= 512) return launch<D, 512, 1>(a, stream);
    if constexpr (D == kF32) {
        if (chunks <= 1024) return launch<D, 1024, 1>(a, stream);
        if (chunks > 2048) return launch<D, 1024, 4>(a, stream);
    } else {
        if (chunks <= 1024) return launch<D, 512, 2>(a, stream);
    }
    return launch<D, 1024, 2>(a, stream);
}

}  // namespace

int64_t backward_workspace(int64_t T, int64_t H) {
    return 4 * 3 * H * std::min<int64_t>(T, most_partials(H));
}

hipError_t launch_backward(const Backward &a, int dtype, hipStream_t stream) {
    switch (dtype) {
        case kBf16: return launch_row<kBf16>(a, stream);
        case kF16: return launch_row<kF16>(a, stream);
        default: return launch_row<kF32>(a, stream);
    }
}

}  // namespace block
