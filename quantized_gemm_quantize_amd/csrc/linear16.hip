// 16-bit products with bias, activation and residual, and their gradients:
// which kernel computes a product, and the pass before the gradients' products.
//
//   forward   pre = x w^T + bias, out = act(pre) + residual
//   backward  d_pre = d_out act'(pre), d_bias = sum_m d_out act'(pre),
//             d_x = d_pre w, d_w = d_pre^T x
//
// d_pre is rounded to the rows' type: it is an operand of the matrix instructions,
// and a result of its own. d_bias is summed from the unrounded values.
#include <algorithm>

#include "activation.hpp"
#include "launch.hpp"
#include "linear16.hpp"
#include "rows.hpp"

namespace linear16 {
namespace {

using namespace rows;

// ---------------------------------------------------------------- plans

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Time of a round of tiles (all that run at once) in us: a fixed part (first loads, epilogue) and a
// part per 64 k, which grows from lo to hi as the chip fills (its power is shared). Measured in HIP
// graphs with bf16 rows of random values, between 1/4 and all of the tiles that run at once, K 512 and 2048.
struct FormTime {
    int bm, bn, slots;          // tiles that run at once on 256 CUs
    double fixed, lo, hi;
};
constexpr FormTime kTimes[kForms] = {
    {64, 64, 768, 3.5, 0.24, 0.53},   // k64x64
    {128, 128, 256, 4.8, 0.40, 0.49}, // k128x128deep
    {128, 128, 512, 4.0, 0.64, 0.90}, // k128x128
    {256, 128, 256, 6.0, 0.63, 0.82}, // k256x128
    {256, 256, 256, 10.0, 1.10, 1.41},// k256x256
    {64, 64, 256, 4.2, 0.12, 0.15}    // k64x64deep
};

double round_time(const FormTime &f, int64_t units, int64_t stages) {
    const double fill = (double)units / f.slots;
    return f.fixed + stages * (f.lo + (f.hi - f.lo) * fill * fill);
}

struct Estimate {
    Plan plan;
    double us;
};

// The plan with the least estimated time: every tile, or all but the last whole rounds' rest, to one
// workgroup; the rest's tiles are shared along k by as many workgroups as run at once (at least
// two stages each), whose partial sums a second launch joins (3 us and their bytes at 4.5 TB/s).
// What splitting the rest is worth: 16448 x 5120 x 1280 (1300 tiles of 256 x 256, 1280 of them in five
// rounds) 218 -> 203 us, 16448 x 1280 x 5120 (325 tiles) 221 -> 207; 64 x 4096 x 8192 (64 tiles of 64 x 64, four
// workgroups each) 37.6 -> 21.7, 300 x 72 x 8200 (10 tiles, twelve each) 34.6 -> 10.5.
Estimate estimate(int64_t M, int64_t N, int64_t K) {
    Estimate best{{k64x64, 0, 1, 0}, -1};
    const int64_t stages = ceil_div(K, 64);
    for (int i = 0; i < kForms; ++i) {
        const FormTime &f = kTimes[i];
        const int64_t tiles = ceil_div(M, f.bm) * ceil_div(N, f.bn), rounds = tiles / f.slots, rest = tiles % f.slots;
        const double whole = rounds * round_time(f, f.slots, stages);
        auto offer = [&](double us, int64_t splits) {
            if (best.us >= 0 && us >= best.us) return;
            const int64_t shared = splits > 1 ? rest : 0;
            best = {{(Form)i, (int)(tiles - shared), (int)splits, shared * splits * f.bm * f.bn * 4}, us};
        };
        offer(whole + (rest ? round_time(f, rest, stages) : 0.0), 1);
        if (!rest) continue;
        const int64_t most = std::min(f.slots / rest, stages / 2);
        for (int64_t s : {2, 3, 4, 6, 8, 12, 16, 24, 32, 64}) {
            s = std::min(s, most);
            if (s < 2) break;
            const double bytes = 2.0 * rest * s * f.bm * f.bn * 4;
            offer(whole + round_time(f, rest * s, ceil_div(stages, s)) + 3.0 + bytes / 4.5e6, s);
            if (s == most) break;
        }
    }
    return best;
}

// The plan with the least estimated time for both gradients in one launch. The product of the longer k goes
// first, its tiles whole or all of them shared by s workgroups; the other's tiles follow on workgroup
// slots as they come free, whole, or whole up to the end of one of their rounds and the rest shared.
// With p slots free from `from` on, q from `later` on (a round of the first product more), and
// `each` a tile: the rounds that hold n tiles, and the tiles done at a time.
PairPlan estimate_pair(int64_t M, int64_t N, int64_t K) {
    const bool w_first = M >= N;
    PairPlan best{{k64x64, (int)(ceil_div(M, 64) * ceil_div(K, 64)), 1, 0}, {k64x64, (int)(ceil_div(N, 64) * ceil_div(K, 64)), 1, 0}, w_first};
    double least = -1;
    // rows, columns and stages of the first product and the second
    const int64_t rows[2] = {w_first ? N : M, w_first ? M : N}, stages[2] = {ceil_div(w_first ? M : N, 64), ceil_div(w_first ? N : M, 64)};
    for (const Form form : {k64x64, k128x128, k256x256}) {
        const FormTime &f = kTimes[form];
        const int64_t columns = ceil_div(K, f.bn), first = ceil_div(rows[0], f.bm) * columns, second = ceil_div(rows[1], f.bm) * columns;
        const double join = 2.0 * f.bm * f.bn * 4 / 4.5e6;   // of one part
        for (int64_t s : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
            if (s > 1 && s > stages[0] / 2) break;
            const int64_t units = first * s, q = units % f.slots, p = f.slots - q;
            const double fill = std::min(1.0, (double)(units + second) / f.slots), per = f.lo + (f.hi - f.lo) * fill * fill;
            const double one = f.fixed + ceil_div(stages[0], s) * per, each = f.fixed + stages[1] * per;
            const double from = units / f.slots * one, later = q ? from + one : from;
            const double joined = s > 1 ? 3.0 + units * join : 0.0, behind = q ? one / each : 0.0;
            auto done = [&](double t) {
                return p * (int64_t)std::max(0.0, (t - from) / each + 1e-9) + q * (int64_t)std::max(0.0, (t - later) / each + 1e-9);
            };
            auto offer = [&](double us, int64_t whole, int64_t splits) {
                if (least >= 0 && us >= least) return;
                least = us;
                const int64_t bytes = (int64_t)f.bm * f.bn * 4;
                const Plan a{form, s > 1 ? 0 : (int)first, (int)s, s > 1 ? units * bytes : 0};
                const Plan b{form, (int)whole, (int)splits, (second - whole) * splits * bytes};
                best = w_first ? PairPlan{b, a, true} : PairPlan{a, b, false};
            };
            // ends after k rounds from `from` on (some before `later`), or from `later` on
            const int64_t early = ceil_div(second, p);
            const int64_t k0 = early <= behind ? early : (int64_t)std::ceil((second + q * std::ceil(behind)) / f.slots);
            const int64_t k1 = std::max<int64_t>(0, ceil_div(second - p * (int64_t)behind, f.slots));
            for (const double end : {from + k0 * each, later + k1 * each}) {
                if (done(end) >= second) offer(std::max(end, later) + joined, second, 1);
                const double before = end - each;
                const int64_t whole = before < later ? 0 : done(before), rest = second - whole;
                if (rest <= 0 || before < later) continue;
                for (int64_t splits : {2, 4, 8, 16, 32}) {
                    if (splits * rest > f.slots || splits > stages[1] / 2) break;
                    offer(before + f.fixed + ceil_div(stages[1], splits) * per + 3.0 + rest * splits * join + joined, whole, splits);
                }
            }
        }
    }
    return best;
}

// Time of the kernel of few rows in us. Up to 16 rows: 3 us and the distinct rows of a workgroup's operands at 55 GB/s a
// round, two workgroups per CU; above: 3 us and 16 rows a tile at 65 GB/s, one per CU.
double rows_time(int64_t M, int64_t N, int64_t K) {
    const int64_t groups = ceil_div(N, 16);
    if (M <= 16) return ceil_div(groups, 512) * (3.0 + 2.0 * K * (std::min<int64_t>(N, 16) + M) / 55e3);
    return ceil_div(groups, 256) * (3.0 + 2.0 * K * 16 * (ceil_div(M, 16) + 1) / 65e3);
}

// The kernel of few rows or, if false, the plan in tiles: the kernel unless tiles are estimated to be quicker, which take
// 3 us and the weight at 4.9 TB/s at least. Over 496 measured sizes that this decides, the choice loses 0.3% of the time
// on average and 20% at most.
//  - Up to 16 rows (rows kernel / tiles, us): a workgroup reads a whole K by itself, so a long one over few channels is
//    shared by tiles (16 x 64 x 16384 18.2 / 9.0, 16 x 256 x 9216 12.6 / 8.4, 16 x 8 x 2^20 1361 / 51, but 16 x 4096 x
//    16384 31.1 / 31.3); many workgroups of a short one pay their start (16 x 32000 x 64 7.6 / 4.1, but x 2048 25.8 /
//    33.5). With up to 8192 inner elements (from 1024 on above 4096 channels) the kernel stays at every size, so that
//    those plans cost the host nothing (two of 0.4 us beside a call of 8). Tiles are the quicker ones there at few
//    channels and the longest K only (16 x 64 x 4096 6.2 / 6.9, 1 x 4096 x 4096 7.7 / 11.7, but 16 x 256 x 8192 10.3 / 7.6, 16
//    x 64 x 8192 10.0 / 8.4), and their second launch takes the host 3 us (calls of 16 x 64 x 8192 10.0 / 11.0).
//  - Up to 64: 24 x 4096 x 4096 10.0 / 12.3, 24 x 4096 x 8192 17.5 / 20.3, 17 x 8192 x 11008 39.5 / 45.8, 64 x 1024 x 1024
//    5.5 / 6.5, 64 x 4096 x 1024 6.0 / 6.6, but 24 x 256 x 8192 13.7 / 8.5, 64 x 4096 x 4096 13.9 / 14.0 (tiles), 64 x
//    8192 x 2048 15.8 / 13.6, 64 x 4096 x 11008 33.3 / 25.9, 64 x 11008 x 4096 36.1 / 25.2.
bool few_rows(int64_t M, int64_t N, int64_t K, Plan &plan) {
    if (M <= 16 && K <= 8192 && (N <= 4096 || K >= 1024)) return true;
    const Estimate tiled = estimate(M, N, K);
    plan = tiled.plan;
    return M <= kMaxRows && rows_time(M, N, K) < std::max(tiled.us, 3.0 + 2.0 * N * K / 4.9e6);
}

// ---------------------------------------------------------------- d_pre and d_bias

// A workgroup takes COLUMNS columns, 8 of them a thread, THREADS / (COLUMNS / 8) rows at a time, every
// G-th turn of the rows, U turns in flight. Column sums are kept in registers, joined with shuffles
// and LDS in a fixed order and left as one partial sum per workgroup, or, with one workgroup for
// all rows, as the result.
template <int A, Dtype D>
__device__ __forceinline__ void slopes(float (&d)[8], uint4 pre) {
    float p[8];
    widen_chunk<D>(pre, p);
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] *= act::slope<A>(p[e]);
}

template <Dtype D, int COLUMNS, int THREADS, int U>
__global__ __launch_bounds__(THREADS) void slope_kernel(const uint16_t *__restrict__ d_out, int64_t ldd,
                                                        const uint16_t *__restrict__ pre, int64_t M, int64_t N, int a,
                                                        uint16_t *__restrict__ d_pre, float *__restrict__ partial) {
    constexpr int PER = COLUMNS / 8, ROWS = THREADS / PER, WAVES = THREADS / kWave;
    static_assert(PER <= kWave, "a wavefront holds whole rows");
    __shared__ float red[WAVES][COLUMNS];
    w8a8::lds_poison(red);
    w8a8::lds_poison_done();
    const int c = threadIdx.x % PER * 8, r = threadIdx.x / PER;
    const int64_t n = (int64_t)blockIdx.x * COLUMNS + c;
    float sum[8] = {};
    if (n < N) {
        const int64_t step = (int64_t)gridDim.y * ROWS;
        for (int64_t m = (int64_t)blockIdx.y * ROWS + r; m < M; m += U * step) {
            uint4 du[U], pu[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = min(m + u * step, M - 1);
                du[u] = w8a8::load16_stream(d_out + row * ldd + n);
                if (a != act::kNone) pu[u] = w8a8::load16_stream(pre + row * N + n);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = m + u * step;
                if (row >= M) break;
                float d[8];
                widen_chunk<D>(du[u], d);
                if (a != act::kNone) {
                    switch (a) {
                        case act::kRelu: slopes<act::kRelu, D>(d, pu[u]); break;
                        case act::kGelu: slopes<act::kGelu, D>(d, pu[u]); break;
                        case act::kGeluTanh: slopes<act::kGeluTanh, D>(d, pu[u]); break;
                        default: slopes<act::kSilu, D>(d, pu[u]); break;
                    }
                    *reinterpret_cast<uint4 *>(d_pre + row * N + n) = narrow_chunk<D>(d);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += d[e];
            }
        }
    }
    if (!partial) return;
#pragma unroll
    for (int off = PER; off < kWave; off <<= 1)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor(sum[e], off, kWave);
    if (threadIdx.x % kWave < PER)
#pragma unroll
        for (int e = 0; e < 8; ++e) red[threadIdx.x / kWave][c + e] = sum[e];
    __syncthreads();
    const int64_t at = (int64_t)blockIdx.x * COLUMNS + threadIdx.x;
    if (threadIdx.x >= COLUMNS || at >= N) return;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) s += red[i][threadIdx.x];
    partial[blockIdx.y * N + at] = s;
}

// d_bias[n] = sum of the G partials of column n: 16 slices in order, then the slices.
constexpr int kSlices = 16;

__global__ __launch_bounds__(64 * kSlices) void sum_kernel(const float *__restrict__ partial, int G, int64_t N,
                                                           float *__restrict__ out) {
    __shared__ float red[kSlices][64];
    w8a8::lds_poison(red);
    w8a8::lds_poison_done();
    const int c = threadIdx.x % 64, slice = threadIdx.x / 64;
    const int64_t n = (int64_t)blockIdx.x * 64 + c;
    float s = 0.0f;
    if (n < N)
#pragma unroll 4
        for (int g = slice; g < G; g += kSlices) s += partial[g * N + n];
    red[slice][c] = s;
    __syncthreads();
    if (slice || n >= N) return;
#pragma unroll
    for (int i = 1; i < kSlices; ++i) s += red[i][c];
    out[n] = s;
}

// Up to kOneGroup rows go to one workgroup of 1024 threads per 16 columns, which needs no partial sums
// (257 x 1040 with 64 columns a workgroup 7.3 us, so 5.4); more to workgroups of 256 threads and 64
// columns, up to 256 beside each other and enough to fill the chip eight times.
constexpr int kOneGroup = 512, kNarrow = 16, kWide = 64, kManyRows = 32;

int sum_groups(int64_t M, int64_t N) {
    if (M <= kOneGroup) return 1;
    return (int)std::min<int64_t>(std::min<int64_t>(ceil_div(M, kManyRows), 256),
                                  std::max<int64_t>(1, 2048 / ceil_div(N, kWide)));
}

int64_t sums_bytes(int64_t M, int64_t N) {
    return M <= kOneGroup ? 0 : (4 * N * sum_groups(M, N) + 255) / 256 * 256;
}

template <Dtype D>
hipError_t launch_slope(const void *d_out, int64_t ldd, const void *pre, int64_t M, int64_t N, int a, void *d_pre,
                        float *d_bias, float *partial, hipStream_t stream) {
    const int G = sum_groups(M, N);
    const uint16_t *d = static_cast<const uint16_t *>(d_out), *p = static_cast<const uint16_t *>(pre);
    uint16_t *to = static_cast<uint16_t *>(d_pre);
    if (M <= kOneGroup) {
        slope_kernel<D, kNarrow, 1024, 1><<<dim3((unsigned)ceil_div(N, kNarrow)), 1024, 0, stream>>>(d, ldd, p, M, N, a, to, d_bias);
        return hipGetLastError();
    }
    slope_kernel<D, kWide, 8 * kManyRows, 4><<<dim3((unsigned)ceil_div(N, kWide), (unsigned)G), 8 * kManyRows, 0, stream>>>(
        d, ldd, p, M, N, a, to, d_bias ? partial : nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !d_bias) return e;
    sum_kernel<<<dim3((unsigned)ceil_div(N, 64)), 64 * kSlices, 0, stream>>>(partial, G, N, d_bias);
    return hipGetLastError();
}

}  // namespace

ForwardPlan plan_forward(int64_t M, int64_t N, int64_t K) {
    ForwardPlan p{};
    p.rows = few_rows(M, N, K, p.tiles);
    return p;
}

// Both gradients, where both are wanted, in one launch: at 24 random sizes whose separate launches were estimated to be
// quicker it took 0.66 to 1.04 of their time (257 x 1040 x 1312 with silu 20.2 -> 14.0 us in all, 3428 x 512 x 4688
// 76.7 -> 59.7, 16448 x 5120 x 1280 525 -> 484; 6 x 3424 x 9600 39.3 -> 40.8).
BackwardPlan plan_backward(int64_t M, int64_t N, int64_t K) {
    BackwardPlan p{};
    p.w = estimate(N, K, M).plan;
    p.workspace = std::max(sums_bytes(M, N), p.w.workspace);   // (the column sums are done before the products)
    if (!M) return p;
    p.x = estimate(M, K, N).plan;
    p.both = estimate_pair(M, N, K);
    p.workspace = std::max({p.workspace, p.x.workspace, p.both.x.workspace + p.both.w.workspace});
    return p;
}

hipError_t launch_forward(const ForwardPlan &plan, const void *x, int64_t ldx, int64_t M, const void *w, int64_t N, int64_t K,
                          bool f16, const Epilogue &ep, void *workspace, hipStream_t stream) {
    if (plan.rows) return launch_rows(x, ldx, (int)M, w, (int)N, (int)K, f16, ep, stream);
    return launch_tiled({x, ldx, false}, {w, K, false}, M, N, K, f16, plan.tiles, static_cast<float *>(workspace), ep, stream);
}

hipError_t launch_backward(const BackwardPlan &plan, const void *d_out, int64_t ldd, const void *x, int64_t ldx, const void *w,
                           const void *pre, int64_t M, int64_t N, int64_t K, bool f16, int a, void *d_pre, void *d_x,
                           void *d_w, float *d_bias, void *workspace, hipStream_t stream) {
    float *const partial = static_cast<float *>(workspace);
    hipError_t e = hipSuccess;
    if (d_bias || (a != act::kNone && M)) {
        e = f16 ? launch_slope<kF16>(d_out, ldd, pre, M, N, a, d_pre, d_bias, partial, stream)
                : launch_slope<kBf16>(d_out, ldd, pre, M, N, a, d_pre, d_bias, partial, stream);
        if (e != hipSuccess) return e;
    }
    const Operand rows{a == act::kNone ? d_out : d_pre, a == act::kNone ? ldd : N, false};
    const Operand weight{w, K, true}, columns{rows.p, rows.ld, true}, inputs{x, ldx, true};
    if (d_x && d_w && M)
        return launch_pair({rows, weight, M, K, N, d_x}, {columns, inputs, N, K, M, d_w}, f16, plan.both, partial, stream);
    auto plain = [](void *out) { return Epilogue{nullptr, nullptr, 0, nullptr, out, act::kNone}; };
    if (d_x && M) e = launch_tiled(rows, weight, M, K, N, f16, plan.x, partial, plain(d_x), stream);
    if (d_w && e == hipSuccess) e = launch_tiled(columns, inputs, N, K, M, f16, plan.w, partial, plain(d_w), stream);
    return e;
}

}  // namespace linear16
