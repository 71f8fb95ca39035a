// Mixture-of-experts routing: tokens sorted by expert and back.
//
// A token t fills `top` slots (t, j), each with an expert id; an id outside
// [0, E) is a slot without an expert (dropped). The slots are sorted by
// expert, stably, the dropped ones last: slot (t, j) becomes row p of the
// sorted arrays, kept as slot_pos[t, j] = p, or ~p (negative) for a dropped
// slot. The rows of expert e are offsets[e] .. offsets[e + 1] - 1.
//
//   gather   rows[p] = x[t]                       (0 for dropped slots)
//   combine  out[t]  = sum_j w[t, j] rows[p(t, j)]  (dropped slots add nothing)
//   and backward: d_x[t] = sum_j d_rows[p], d_rows[p] = w[t, j] d_out[t],
//   d_w[t, j] = <d_out[t], rows[p]>.
//
// Sums run in fp32 in the order of j (and a fixed tree over the row), so
// results do not depend on how the work is spread. All of it is bound by HBM.
#include <type_traits>

#include "launch.hpp"
#include "mxfp4.hpp"

namespace moe {
namespace {

using w8a8::kWave;
using mxfp4::Dtype;
using mxfp4::kBf16;
using mxfp4::kF16;
using mxfp4::kF32;

// ------------------------------------------------------------------ sort

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kSortIters = 4;                               // slots per thread
constexpr int kChunk = kSortThreads * kSortIters;           // slots per workgroup
constexpr int kMaxBins = 513;                               // experts, and the dropped slots

template <typename I>
__device__ __forceinline__ int bin_of(const I *ids, int64_t slot, int64_t S, int E) {
    if (slot >= S) return -1;
    const I id = ids[slot];
    return id >= 0 && id < (I)E ? (int)id : E;
}

// The lanes of the wavefront that hold the same bin (-1: none).
__device__ __forceinline__ uint64_t same_bin(int bin, int bits) {
    uint64_t m = __builtin_amdgcn_ballot_w64(bin >= 0);
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __builtin_amdgcn_ballot_w64((bin >> b) & 1);
        m &= (bin >> b) & 1 ? set : ~set;
    }
    return m;
}

// Each workgroup counts the bins of its kChunk slots.
template <typename I>
__global__ __launch_bounds__(kSortThreads) void count_kernel(const I *__restrict__ ids, int64_t S,
                                                             int E, int32_t *__restrict__ counts) {
    __shared__ int hist[kMaxBins + 3];
    w8a8::lds_poison(hist);
    w8a8::lds_poison_done();
    for (int e = threadIdx.x; e <= E; e += kSortThreads) hist[e] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSortIters; ++i) {
        const int64_t slot = (int64_t)blockIdx.x * kChunk + i * kSortThreads + threadIdx.x;
        const int bin = bin_of(ids, slot, S, E);
        if (bin >= 0) atomicAdd(&hist[bin], 1);  // integers: the order does not matter
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kSortThreads)
        counts[(int64_t)blockIdx.x * (E + 1) + e] = hist[e];
}

// Places the slots of one chunk. Wavefront w owns slots [w * 64 * kSortIters,
// +64 * kSortIters) of the chunk; a slot's row is the bin's first row, plus
// the bin's slots in earlier chunks (counts), in earlier wavefronts, and
// before it in its own wavefront (lane order within a match mask): the stable
// order. With one chunk the counts are this workgroup's own.
template <typename I>
__global__ __launch_bounds__(kSortThreads) void place_kernel(
    const I *__restrict__ ids, int64_t S, int top, int E, int bits,
    const int32_t *__restrict__ counts, int chunks, int32_t *__restrict__ offsets,
    int32_t *__restrict__ slot_pos, int32_t *__restrict__ row_token) {
    extern __shared__ int hist[];  // [kSortWaves][E + 1] counts, then first rows
    __shared__ int wave_sum[kSortWaves];
    const int bins = E + 1;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    w8a8::lds_poison(wave_sum);
    w8a8::lds_poison_done();
    for (int i = threadIdx.x; i < kSortWaves * bins; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    int bin[kSortIters], before[kSortIters];
    const int64_t first = (int64_t)blockIdx.x * kChunk + wave * (kWave * kSortIters) + lane;
#pragma unroll
    for (int i = 0; i < kSortIters; ++i) bin[i] = bin_of(ids, first + i * kWave, S, E);
#pragma unroll
    for (int i = 0; i < kSortIters; ++i) {
        const uint64_t same = same_bin(bin[i], bits);
        const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
        int *h = hist + wave * bins + bin[i];
        before[i] = 0;
        if (bin[i] >= 0) before[i] = *h + rank;
        // the last lane of a bin carries its count on (one writer per bin)
        if (bin[i] >= 0 && (same >> lane) == 1) *h = before[i] + 1;
        asm volatile("" ::: "memory");
    }
    __syncthreads();
    // per bin (thread e): the wavefronts' starts, the slots in earlier chunks,
    // all slots
    const int e = threadIdx.x;
    int total = 0, earlier = 0;
    if (e < bins) {
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = hist[w * bins + e];
            hist[w * bins + e] = total;
            total += c;
        }
        if (chunks > 1) {
            total = 0;
            for (int c = 0; c < chunks; ++c) {
                const int v = counts[(int64_t)c * bins + e];
                if (c < (int)blockIdx.x) earlier += v;
                total += v;
            }
        }
    }
    // first row of each bin: an exclusive scan of the totals over the threads
    int upto = total;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const int o = __shfl_up(upto, off, kWave);
        if (lane >= off) upto += o;
    }
    if (lane == kWave - 1) wave_sum[wave] = upto;
    __syncthreads();
    int start = upto - total;
    for (int w = 0; w < wave; ++w) start += wave_sum[w];
    if (e < bins) {
        for (int w = 0; w < kSortWaves; ++w) hist[w * bins + e] += start + earlier;
        if (blockIdx.x == 0) offsets[e] = start;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSortIters; ++i) {
        if (bin[i] < 0) continue;
        const int64_t slot = first + i * kWave;
        const int p = hist[wave * bins + bin[i]] + before[i];
        const bool kept = bin[i] < E;
        slot_pos[slot] = kept ? p : ~p;
        row_token[p] = kept ? (int)((uint32_t)slot / (uint32_t)top) : -1;
    }
}

// ------------------------------------------------------------------ rows

constexpr int kThreads = 256;

// V elements of a row as floats. V > 1: one 16-byte access.
template <Dtype D, int V>
__device__ __forceinline__ void load_row(const char *p, float (&f)[V]) {
    if constexpr (V == 1) {
        if constexpr (D == kF32) f[0] = *reinterpret_cast<const float *>(p);
        else if constexpr (D == kBf16) f[0] = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(p) << 16);
        else f[0] = (float)*reinterpret_cast<const _Float16 *>(p);
    } else {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (D == kF32) f[i] = __uint_as_float(w[i]);
            else if constexpr (D == kBf16) { f[2 * i] = w8a8::bf16_lo(w[i]); f[2 * i + 1] = w8a8::bf16_hi(w[i]); }
            else { const mxfp4::v2h h = __builtin_bit_cast(mxfp4::v2h, w[i]); f[2 * i] = (float)h[0]; f[2 * i + 1] = (float)h[1]; }
        }
    }
}

template <Dtype D, int V>
__device__ __forceinline__ void store_row(char *p, const float (&f)[V]) {
    if constexpr (V == 1) {
        if constexpr (D == kF32) *reinterpret_cast<float *>(p) = f[0];
        else if constexpr (D == kBf16) *reinterpret_cast<__bf16 *>(p) = (__bf16)f[0];
        else *reinterpret_cast<_Float16 *>(p) = (_Float16)f[0];
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (D == kF32) w[i] = __float_as_uint(f[i]);
            else if constexpr (D == kBf16) w[i] = w8a8::pack_bf16x2(f[2 * i], f[2 * i + 1]);
            else w[i] = __builtin_bit_cast(uint32_t, mxfp4::v2h{(_Float16)f[2 * i], (_Float16)f[2 * i + 1]});
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <Dtype D>
constexpr int size_of() { return D == kF32 ? 4 : 2; }

// Row of slot_pos value p, kept or dropped; -1 when a malformed plan points
// outside the S rows.
__device__ __forceinline__ int64_t row_of(int p, int64_t S) {
    const int64_t r = p < 0 ? ~(int64_t)p : p;
    return r < S ? r : -1;
}

// One workgroup: a token, kThreads * V of its elements. Each element is read
// once and written to all of the token's rows.
template <Dtype D, int V>
__global__ __launch_bounds__(kThreads) void gather_kernel(const char *__restrict__ x, int64_t ldx,
                                                          const int32_t *__restrict__ slot_pos,
                                                          int top, int64_t S, int H,
                                                          char *__restrict__ rows) {
    const int64_t t = blockIdx.x;
    const int h = (blockIdx.y * kThreads + threadIdx.x) * V;
    if (h >= H) return;
    float f[V], zero[V] = {};
    load_row<D, V>(x + (t * ldx + h) * size_of<D>(), f);
    for (int j = 0; j < top; ++j) {
        const int p = slot_pos[t * top + j];
        const int64_t r = row_of(p, S);
        if (r < 0) continue;
        store_row<D, V>(rows + (r * H + h) * size_of<D>(), p < 0 ? zero : f);
    }
}

template <Dtype D, int V, bool WEIGHTS>
__global__ __launch_bounds__(kThreads) void combine_kernel(const char *__restrict__ rows,
                                                           const int32_t *__restrict__ slot_pos,
                                                           const float *__restrict__ weights,
                                                           int top, int64_t S, int H,
                                                           char *__restrict__ out) {
    const int64_t t = blockIdx.x;
    const int h = (blockIdx.y * kThreads + threadIdx.x) * V;
    if (h >= H) return;
    float sum[V] = {};
    for (int j = 0; j < top; ++j) {
        const int p = slot_pos[t * top + j];
        if (p < 0 || p >= S) continue;
        const float w = WEIGHTS ? weights[t * top + j] : 1.0f;
        float f[V];
        load_row<D, V>(rows + ((int64_t)p * H + h) * size_of<D>(), f);
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] += WEIGHTS ? w * f[i] : f[i];
    }
    store_row<D, V>(out + (t * H + h) * size_of<D>(), sum);
}

// One workgroup per token: d_rows, and d_w summed over the row (each thread
// its elements in order, then lanes, then wavefronts).
template <Dtype D, int V>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(
    const char *__restrict__ d_out, int64_t ldd, const char *__restrict__ rows,
    const int32_t *__restrict__ slot_pos, const float *__restrict__ weights, int top, int64_t S,
    int H, char *__restrict__ d_rows, float *__restrict__ d_weights) {
    __shared__ float part[kThreads / kWave];
    w8a8::lds_poison(part);
    w8a8::lds_poison_done();
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    for (int j = 0; j < top; ++j) {
        const int p = slot_pos[t * top + j];
        const int64_t r = row_of(p, S);
        const bool kept = p >= 0 && r >= 0;
        const float w = kept ? weights[t * top + j] : 0.0f;
        float dot = 0.0f;
        for (int h = threadIdx.x * V; h < H; h += kThreads * V) {
            float d[V], g[V] = {};
            if (kept) {
                float y[V];
                load_row<D, V>(d_out + (t * ldd + h) * size_of<D>(), d);
                load_row<D, V>(rows + (r * H + h) * size_of<D>(), y);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    g[i] = w * d[i];
                    dot += d[i] * y[i];
                }
            }
            if (r >= 0) store_row<D, V>(d_rows + (r * H + h) * size_of<D>(), g);
        }
        if (d_weights) {
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) dot += __shfl_xor(dot, off, kWave);
            if (lane == 0) part[wave] = dot;
            __syncthreads();
            if (threadIdx.x == 0) d_weights[t * top + j] = kept ? part[0] + part[1] + part[2] + part[3] : 0.0f;
            __syncthreads();
        }
    }
}

// 16-byte accesses when every row starts 16-byte aligned.
bool wide(const void *a, const void *b, const void *c, int64_t ld, int64_t H, int dtype) {
    const int64_t size = dtype == kF32 ? 4 : 2;
    const uintptr_t p = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) |
                        reinterpret_cast<uintptr_t>(c);
    return (p & 15) == 0 && H * size % 16 == 0 && ld * size % 16 == 0;
}

int segments(int H, int per_thread) { return (H + kThreads * per_thread - 1) / (kThreads * per_thread); }

// f(Dtype constant, elements per access)
template <typename F>
void by_type(int dtype, bool w, F f) {
    using std::integral_constant;
    switch (dtype) {
        case kBf16: w ? f(integral_constant<Dtype, kBf16>{}, integral_constant<int, 8>{}) : f(integral_constant<Dtype, kBf16>{}, integral_constant<int, 1>{}); break;
        case kF16: w ? f(integral_constant<Dtype, kF16>{}, integral_constant<int, 8>{}) : f(integral_constant<Dtype, kF16>{}, integral_constant<int, 1>{}); break;
        default: w ? f(integral_constant<Dtype, kF32>{}, integral_constant<int, 4>{}) : f(integral_constant<Dtype, kF32>{}, integral_constant<int, 1>{});
    }
}

template <typename I>
hipError_t sort_ids(const I *ids, int64_t S, int top, int E, int32_t *offsets, int32_t *slot_pos,
                    int32_t *row_token, int32_t *counts, hipStream_t stream) {
    const int chunks = S > 0 ? (int)((S + kChunk - 1) / kChunk) : 1;  // none: offsets only
    int bits = 0;
    while ((1 << bits) <= E) ++bits;
    if (chunks > 1) {
        count_kernel<I><<<chunks, kSortThreads, 0, stream>>>(ids, S, E, counts);
        if (hipError_t e = hipGetLastError()) return e;
    }
    place_kernel<I><<<chunks, kSortThreads, kSortWaves * (E + 1) * sizeof(int), stream>>>(
        ids, S, top, E, bits, counts, chunks, offsets, slot_pos, row_token);
    return hipGetLastError();
}

}  // namespace

int64_t sort_workspace(int64_t S, int64_t E) {
    const int64_t chunks = (S + kChunk - 1) / kChunk;
    return chunks > 1 ? chunks * (E + 1) * (int64_t)sizeof(int32_t) : 0;
}

hipError_t launch_sort(const void *ids, bool ids64, int64_t S, int top, int E, int32_t *offsets,
                       int32_t *slot_pos, int32_t *row_token, void *workspace, hipStream_t stream) {
    int32_t *counts = static_cast<int32_t *>(workspace);
    if (ids64)
        return sort_ids(static_cast<const int64_t *>(ids), S, top, E, offsets, slot_pos, row_token, counts, stream);
    return sort_ids(static_cast<const int32_t *>(ids), S, top, E, offsets, slot_pos, row_token, counts, stream);
}

hipError_t launch_gather(const void *x, int64_t ldx, const int32_t *slot_pos, int64_t T, int top,
                         int H, int dtype, void *rows, hipStream_t stream) {
    by_type(dtype, wide(x, rows, nullptr, ldx, H, dtype), [&](auto d, auto v) {
        gather_kernel<decltype(d)::value, decltype(v)::value>
            <<<dim3((unsigned)T, segments(H, v)), kThreads, 0, stream>>>(
                static_cast<const char *>(x), ldx, slot_pos, top, T * top, H, static_cast<char *>(rows));
    });
    return hipGetLastError();
}

hipError_t launch_combine(const void *rows, const int32_t *slot_pos, const float *weights,
                          int64_t T, int top, int H, int dtype, void *out, hipStream_t stream) {
    by_type(dtype, wide(rows, out, nullptr, H, H, dtype), [&](auto d, auto v) {
        const dim3 grid((unsigned)T, segments(H, v));
        const char *r = static_cast<const char *>(rows);
        char *o = static_cast<char *>(out);
        if (weights)
            combine_kernel<decltype(d)::value, decltype(v)::value, true>
                <<<grid, kThreads, 0, stream>>>(r, slot_pos, weights, top, T * top, H, o);
        else
            combine_kernel<decltype(d)::value, decltype(v)::value, false>
                <<<grid, kThreads, 0, stream>>>(r, slot_pos, weights, top, T * top, H, o);
    });
    return hipGetLastError();
}

hipError_t launch_combine_backward(const void *d_out, int64_t ldd, const void *rows,
                                   const int32_t *slot_pos, const float *weights, int64_t T,
                                   int top, int H, int dtype, void *d_rows, float *d_weights,
                                   hipStream_t stream) {
    by_type(dtype, wide(d_out, rows, d_rows, ldd, H, dtype), [&](auto d, auto v) {
        combine_backward_kernel<decltype(d)::value, decltype(v)::value>
            <<<dim3((unsigned)T), kThreads, 0, stream>>>(
                static_cast<const char *>(d_out), ldd, static_cast<const char *>(rows), slot_pos,
                weights, top, T * top, H, static_cast<char *>(d_rows), d_weights);
    });
    return hipGetLastError();
}

}  // namespace moe
