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
// results do not depend on how the work is spread. The rows' kernels are bound
// by HBM and go token by token, so that each token is read once. Measured, 16448
// tokens x 4 slots x 4096 bf16: gather 121 us (674 MB, 5.6 TB/s), combine 111 (6.1),
// its backward 232 (1.21 GB, 5.2), the gather's 111; rows that are no multiple of 16
// bytes: 4098 elements gather 239, combine 165, backward 389, 4095 195, 132, 407. The sum
// of a layer's fp32 rows, 8192 tokens x 4, 100 (604 MB, 6.0). The sort of the 65792
// slots, bound by the latency of its two launches, 12, of 16.8 million 128 (three).
#include <type_traits>

#include "launch.hpp"
#include "mxfp4_rows.hpp"

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
constexpr int kSums = 12;                                   // chunks that a thread sums, see sort_ids
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

// Rows that are quantized to MXFP4 by the workgroups after the sort's own, in
// the same launch (codes null: none).
struct Rows {
    const char *x;
    int64_t ldx, M;
    int K, KB;
    uint8_t *codes, *scales;
};

template <int QD>
__device__ __forceinline__ void quantize_beside(int64_t block, const Rows &q) {
    if constexpr (QD >= 0)
        mxfp4::quantize_steps<(Dtype)QD, 1, kSortThreads>(block, q.x, q.ldx, q.M, q.K, q.KB, q.codes, q.scales);
}

// Each workgroup counts the bins of its kChunk slots.
template <typename I, int QD>
__global__ __launch_bounds__(kSortThreads) void count_kernel(const I *__restrict__ ids, int64_t S,
                                                             int E, int32_t *__restrict__ counts,
                                                             int chunks, Rows q) {
    if (QD >= 0 && (int)blockIdx.x >= chunks) return quantize_beside<QD>(blockIdx.x - chunks, q);
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

// Many chunks: workgroup e turns bin e's counts into the bin's slots in earlier
// chunks, and leaves its slots in all chunks behind them (`counts` has chunks + 1
// rows then).
__global__ __launch_bounds__(kSortThreads) void scan_kernel(int32_t *__restrict__ counts, int chunks, int bins) {
    __shared__ int wave_sum[kSortWaves];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    w8a8::lds_poison(wave_sum);
    w8a8::lds_poison_done();
    int before = 0;
    for (int base = 0; base < chunks; base += kSortThreads) {
        const int c = base + threadIdx.x;
        int32_t *at = counts + (int64_t)c * bins + blockIdx.x;
        const int own = c < chunks ? *at : 0;
        int upto = own;
#pragma unroll
        for (int off = 1; off < kWave; off <<= 1) {
            const int o = __shfl_up(upto, off, kWave);
            if (lane >= off) upto += o;
        }
        if (lane == kWave - 1) wave_sum[wave] = upto;
        __syncthreads();
        int all = 0, earlier = before;
        for (int w = 0; w < kSortWaves; ++w) {
            if (w < wave) earlier += wave_sum[w];
            all += wave_sum[w];
        }
        if (c < chunks) *at = earlier + upto - own;
        before += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) counts[(int64_t)chunks * bins + blockIdx.x] = before;
}

// Places the slots of one chunk. Wavefront w owns slots [w * 64 * kSortIters,
// +64 * kSortIters) of the chunk; a slot's row is the bin's first row, plus
// the bin's slots in earlier chunks (counts), in earlier wavefronts, and
// before it in its own wavefront (lane order within a match mask): the stable
// order. With one chunk the counts are this workgroup's own, with several each
// workgroup sums them, and with many the scan has (SCANNED).
template <typename I, int QD, bool SCANNED>
__global__ __launch_bounds__(kSortThreads) void place_kernel(
    const I *__restrict__ ids, int64_t S, int top, int E, int bits,
    const int32_t *__restrict__ counts, int chunks, int32_t *__restrict__ offsets,
    int32_t *__restrict__ slot_pos, int32_t *__restrict__ row_token, Rows q) {
    if (QD >= 0 && (int)blockIdx.x >= chunks) return quantize_beside<QD>(blockIdx.x - chunks, q);
    extern __shared__ int hist[];  // [kSortWaves][E + 1] counts, then first rows; [2][E + 1] sums over chunks
    __shared__ int wave_sum[kSortWaves];
    const int bins = E + 1;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    w8a8::lds_poison(wave_sum);
    w8a8::lds_poison_done();
    int *sums = hist + kSortWaves * bins;
    for (int i = threadIdx.x; i < (kSortWaves + 2) * bins; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    if (!SCANNED && chunks > 1) {
        // as many threads per bin as there are, each with every parts-th chunk
        const int parts = kSortThreads / bins, b = threadIdx.x % bins;
        int before = 0, all = 0;
        for (int c = threadIdx.x / bins; c < chunks && threadIdx.x < parts * bins; c += parts) {
            const int v = counts[(int64_t)c * bins + b];
            if (c < (int)blockIdx.x) before += v;
            all += v;
        }
        if (before) atomicAdd(&sums[b], before);  // integers: the order does not matter
        if (all) atomicAdd(&sums[bins + b], all);
    }
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
        if constexpr (SCANNED) {
            earlier = counts[(int64_t)blockIdx.x * bins + e];
            total = counts[(int64_t)chunks * bins + e];
        } else if (chunks > 1) {
            earlier = sums[e];
            total = sums[bins + e];
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
constexpr int kSlots = 4;  // slots of a token whose rows are in flight together

template <Dtype D>
constexpr int size_of() { return D == kF32 ? 4 : 2; }

typedef uint32_t v2u32 __attribute__((ext_vector_type(2)));

// V elements of a row, as loaded: 16 bytes (V * size = 16), 8, 4 bytes, or one
// element. Everything here is read once and written once: streaming accesses.
template <Dtype D, int V>
struct Vec {
    static constexpr int kBytes = V * size_of<D>();
    static_assert(kBytes == 16 || kBytes == 8 || kBytes == 4 || V == 1, "one access");
    static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const char *p) {
        static_assert(kBytes != 8, "8 bytes are only written");
        if constexpr (kBytes == 16) {
            const uint4 u = w8a8::load16_stream(p);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else if constexpr (kBytes == 4) {
            w[0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(p));
        } else {
            w[0] = __builtin_nontemporal_load(reinterpret_cast<const uint16_t *>(p));
        }
    }
    __device__ __forceinline__ void store(char *p) const {
        if constexpr (kBytes == 16) w8a8::store16_nt(p, make_uint4(w[0], w[1], w[2], w[3]));
        else if constexpr (kBytes == 8)
            __builtin_nontemporal_store(__builtin_bit_cast(v2u32, make_uint2(w[0], w[1])), reinterpret_cast<v2u32 *>(p));
        else if constexpr (kBytes == 4) __builtin_nontemporal_store(w[0], reinterpret_cast<uint32_t *>(p));
        else __builtin_nontemporal_store((uint16_t)w[0], reinterpret_cast<uint16_t *>(p));
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (D == kF32) return __uint_as_float(w[i]);
        else if constexpr (D == kBf16) return i & 1 ? w8a8::bf16_hi(w[i / 2]) : w8a8::bf16_lo(w[i / 2]);
        else return (float)__builtin_bit_cast(mxfp4::v2h, w[i / 2])[i & 1];
    }
    __device__ __forceinline__ void set(const float (&f)[V]) {
        if constexpr (D == kF32) {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __float_as_uint(f[i]);
        } else {
#pragma unroll
            for (int i = 0; i < (V + 1) / 2; ++i) {
                const float lo = f[2 * i], hi = 2 * i + 1 < V ? f[2 * i + 1] : 0.0f;
                if constexpr (D == kBf16) w[i] = w8a8::pack_bf16x2(lo, hi);
                else w[i] = __builtin_bit_cast(uint32_t, mxfp4::v2h{(_Float16)lo, (_Float16)hi});
            }
        }
    }
};

// Row of slot_pos value p, kept or dropped; -1 when a malformed plan points
// outside the S rows.
__device__ __forceinline__ int64_t row_of(int p, int64_t S) {
    const int64_t r = p < 0 ? ~(int64_t)p : p;
    return r < S ? r : -1;
}

// One workgroup: a token, U pieces of kThreads * V of its elements. Each element
// is read once and written to all of the token's rows.
template <Dtype D, int V, int U>
__global__ __launch_bounds__(kThreads) void gather_kernel(const char *__restrict__ x, int64_t ldx,
                                                          const int32_t *__restrict__ slot_pos,
                                                          int top, int64_t S, int H,
                                                          char *__restrict__ rows) {
    const int64_t t = blockIdx.x;
    const int h0 = (blockIdx.y * U * kThreads + threadIdx.x) * V;
    Vec<D, V> v[U], zero;
    zero.clear();
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (h0 + u * kThreads * V < H) v[u].load(x + (t * ldx + h0 + u * kThreads * V) * size_of<D>());
    for (int j = 0; j < top; ++j) {
        const int p = slot_pos[t * top + j];
        const int64_t r = row_of(p, S);
        if (r < 0) continue;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (h0 + u * kThreads * V < H)
                (p < 0 ? zero : v[u]).store(rows + (r * H + h0 + u * kThreads * V) * size_of<D>());
    }
}

// A row's value in the sum of a layer of type D whose rows are held in fp32. Binary16
// layers give what their products and sums give one by one, to the bit: the value has
// binary16's precision, but where that type has no finite value for it it stays as it is
// (an expert's output may lie past 65504 while the weighted sum does not).
template <Dtype D, Dtype R>
__device__ __forceinline__ float row_value(float v) {
    if constexpr (D == kF16 && R == kF32) return fabsf(v) < 65520.0f ? (float)(_Float16)v : v;
    else return v;
}

// The token's rows (type R), kSlots of them in flight together, summed in the order
// of its slots.
template <Dtype D, Dtype R, int V, int U, bool WEIGHTS>
__global__ __launch_bounds__(kThreads) void combine_kernel(const char *__restrict__ rows,
                                                           const int32_t *__restrict__ slot_pos,
                                                           const float *__restrict__ weights,
                                                           int top, int64_t S, int H,
                                                           char *__restrict__ out) {
    const int64_t t = blockIdx.x;
    const int h0 = (blockIdx.y * U * kThreads + threadIdx.x) * V;
    float sum[U][V] = {};
    for (int j0 = 0; j0 < top; j0 += kSlots) {
        Vec<R, V> v[kSlots][U];
        float w[kSlots];
        bool kept[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            const int64_t s = t * top + min(j0 + j, top - 1);
            const int p = slot_pos[s];
            w[j] = WEIGHTS ? weights[s] : 1.0f;
            kept[j] = j0 + j < top && p >= 0 && p < S;
            if (kept[j]) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (h0 + u * kThreads * V < H)
                        v[j][u].load(rows + ((int64_t)p * H + h0 + u * kThreads * V) * size_of<R>());
            }
        }
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            if (!kept[j]) continue;  // uniform
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float y = row_value<D, R>(v[j][u].get(i));
                    sum[u][i] += WEIGHTS ? w[j] * y : y;
                }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (h0 + u * kThreads * V < H) {
            Vec<D, V> v;
            v.set(sum[u]);
            v.store(out + (t * H + h0 + u * kThreads * V) * size_of<D>());
        }
}

// One workgroup per token: d_rows, and d_weights summed over the row (each
// thread its elements in order, then lanes, then wavefronts). kSlots slots
// together: d_out is read once for them, their sums are joined together.
template <Dtype D, int V>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(
    const char *__restrict__ d_out, int64_t ldd, const char *__restrict__ rows,
    const int32_t *__restrict__ slot_pos, const float *__restrict__ weights, int top, int64_t S,
    int H, char *__restrict__ d_rows, float *__restrict__ d_weights) {
    constexpr int kWaves = kThreads / kWave;
    __shared__ float part[kSlots][kWaves];
    w8a8::lds_poison(part);
    w8a8::lds_poison_done();
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    for (int j0 = 0; j0 < top; j0 += kSlots) {
        int64_t row[kSlots];
        bool kept[kSlots];
        float w[kSlots], dot[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            const int64_t s = t * top + min(j0 + j, top - 1);
            const int p = slot_pos[s];
            row[j] = j0 + j < top ? row_of(p, S) : -1;
            kept[j] = p >= 0 && row[j] >= 0;
            w[j] = weights[s];
            dot[j] = 0.0f;
        }
        for (int h = threadIdx.x * V; h < H; h += kThreads * V) {
            Vec<D, V> d, y[kSlots];
            d.load(d_out + (t * ldd + h) * size_of<D>());
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (kept[j]) y[j].load(rows + (row[j] * H + h) * size_of<D>());
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                if (row[j] < 0) continue;  // uniform, as kept
                float g[V] = {};
                if (kept[j]) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        g[i] = w[j] * d.get(i);
                        dot[j] += d.get(i) * y[j].get(i);
                    }
                }
                Vec<D, V> v;
                v.set(g);
                v.store(d_rows + (row[j] * H + h) * size_of<D>());
            }
        }
        if (d_weights) {
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
#pragma unroll
                for (int off = 32; off > 0; off >>= 1) dot[j] += __shfl_xor(dot[j], off, kWave);
                if (lane == 0) part[j][wave] = dot[j];
            }
            __syncthreads();
            if (threadIdx.x < kSlots && j0 + (int)threadIdx.x < top) {
                const int j = threadIdx.x;
                bool k = false;
#pragma unroll
                for (int q = 0; q < kSlots; ++q)
                    if (q == j) k = kept[q];
                float sum = 0.0f;
#pragma unroll
                for (int q = 0; q < kWaves; ++q) sum += part[j][q];
                d_weights[t * top + j0 + j] = k ? sum : 0.0f;
            }
            __syncthreads();
        }
    }
}

// Bytes per access: 16 or 4 when every row starts aligned to that, else one
// element.
int access(const void *a, const void *b, const void *c, int64_t ld, int64_t H, int dtype) {
    const int64_t size = dtype == kF32 ? 4 : 2;
    const uint64_t p = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) |
                       reinterpret_cast<uintptr_t>(c) | (uint64_t)(H * size) | (uint64_t)(ld * size);
    return p % 16 == 0 ? 16 : p % 4 == 0 ? 4 : 2;
}

// f(Dtype constant, elements per access)
template <typename F>
void by_type(int dtype, int bytes, F f) {
    using std::integral_constant;
    if (dtype == kF32) {
        const integral_constant<Dtype, kF32> d;
        bytes == 16 ? f(d, integral_constant<int, 4>{}) : f(d, integral_constant<int, 1>{});
    } else if (dtype == kBf16) {
        const integral_constant<Dtype, kBf16> d;
        bytes == 16 ? f(d, integral_constant<int, 8>{})
                    : bytes == 4 ? f(d, integral_constant<int, 2>{}) : f(d, integral_constant<int, 1>{});
    } else {
        const integral_constant<Dtype, kF16> d;
        bytes == 16 ? f(d, integral_constant<int, 8>{})
                    : bytes == 4 ? f(d, integral_constant<int, 2>{}) : f(d, integral_constant<int, 1>{});
    }
}

// Elements per thread: one 16-byte access, or four short ones (fewer bytes in
// flight per thread would not fill the memory's latency).
template <typename V>
constexpr int unroll() { return V::value * 2 >= 8 ? 1 : 4; }

int segments(int H, int per_thread) { return (H + kThreads * per_thread - 1) / (kThreads * per_thread); }

template <typename I, int QD>
hipError_t sort_ids(const I *ids, int64_t S, int top, int E, int32_t *offsets, int32_t *slot_pos,
                    int32_t *row_token, int32_t *counts, const Rows &q, hipStream_t stream) {
    const int chunks = S > 0 ? (int)((S + kChunk - 1) / kChunk) : 1;  // none: offsets only
    int bits = 0;
    while ((1 << bits) <= E) ++bits;
    const int steps_per_block = kSortThreads / 32;
    const int beside = QD >= 0 ? (int)((q.M * q.KB + steps_per_block - 1) / steps_per_block) : 0;
    const size_t lds = (kSortWaves + 2) * (E + 1) * sizeof(int);
    if (chunks == 1) {
        place_kernel<I, QD, false><<<chunks + beside, kSortThreads, lds, stream>>>(ids, S, top, E, bits, counts, chunks,
                                                                                   offsets, slot_pos, row_token, q);
        return hipGetLastError();
    }
    count_kernel<I, QD><<<chunks + beside, kSortThreads, 0, stream>>>(ids, S, E, counts, chunks, q);
    if (hipError_t e = hipGetLastError()) return e;
    // Every workgroup sums the chunks, kSortThreads / bins threads per bin, or a
    // scan of its own launch does (us: 17 chunks of 64 experts 14.5 with a thread
    // per bin, 10.9 with 15; 512 experts, 59 chunks 26.4 so, 16 scanned; 512 chunks of
    // 64 experts 133, 23.4 scanned).
    if ((int64_t)chunks * (E + 1) <= kSums * kSortThreads) {
        place_kernel<I, -1, false><<<chunks, kSortThreads, lds, stream>>>(ids, S, top, E, bits, counts, chunks, offsets,
                                                                          slot_pos, row_token, q);
        return hipGetLastError();
    }
    scan_kernel<<<E + 1, kSortThreads, 0, stream>>>(counts, chunks, E + 1);
    if (hipError_t e = hipGetLastError()) return e;
    place_kernel<I, -1, true><<<chunks, kSortThreads, lds, stream>>>(ids, S, top, E, bits, counts, chunks, offsets,
                                                                     slot_pos, row_token, q);
    return hipGetLastError();
}

template <int QD>
hipError_t sort_any(const void *ids, bool ids64, int64_t S, int top, int E, int32_t *offsets,
                    int32_t *slot_pos, int32_t *row_token, void *workspace, const Rows &q,
                    hipStream_t stream) {
    int32_t *counts = static_cast<int32_t *>(workspace);
    if (ids64)
        return sort_ids<int64_t, QD>(static_cast<const int64_t *>(ids), S, top, E, offsets, slot_pos, row_token, counts, q, stream);
    return sort_ids<int32_t, QD>(static_cast<const int32_t *>(ids), S, top, E, offsets, slot_pos, row_token, counts, q, stream);
}

}  // namespace

int64_t sort_workspace(int64_t S, int64_t E) {
    const int64_t chunks = (S + kChunk - 1) / kChunk;
    return chunks > 1 ? (chunks + 1) * (E + 1) * (int64_t)sizeof(int32_t) : 0;
}

hipError_t launch_sort(const void *ids, bool ids64, int64_t S, int top, int E, int32_t *offsets,
                       int32_t *slot_pos, int32_t *row_token, void *workspace, hipStream_t stream) {
    return sort_any<-1>(ids, ids64, S, top, E, offsets, slot_pos, row_token, workspace, Rows{}, stream);
}

hipError_t launch_sort_quantize(const void *ids, bool ids64, int64_t S, int top, int E,
                                int32_t *offsets, int32_t *slot_pos, int32_t *row_token,
                                void *workspace, const void *x, int64_t ldx, int64_t T, int H,
                                int dtype, uint8_t *codes, uint8_t *scales, hipStream_t stream) {
    const Rows q{static_cast<const char *>(x), ldx, T, H, (H + mxfp4::kStep - 1) / mxfp4::kStep, codes, scales};
    switch (dtype) {
        case kBf16: return sort_any<kBf16>(ids, ids64, S, top, E, offsets, slot_pos, row_token, workspace, q, stream);
        case kF16: return sort_any<kF16>(ids, ids64, S, top, E, offsets, slot_pos, row_token, workspace, q, stream);
        default: return sort_any<kF32>(ids, ids64, S, top, E, offsets, slot_pos, row_token, workspace, q, stream);
    }
}

hipError_t launch_gather(const void *x, int64_t ldx, const int32_t *slot_pos, int64_t T, int top,
                         int H, int dtype, void *rows, hipStream_t stream) {
    by_type(dtype, access(x, rows, nullptr, ldx, H, dtype), [&](auto d, auto v) {
        constexpr int V = decltype(v)::value, U = unroll<decltype(v)>();
        gather_kernel<decltype(d)::value, V, U><<<dim3((unsigned)T, segments(H, V * U)), kThreads, 0, stream>>>(
            static_cast<const char *>(x), ldx, slot_pos, top, T * top, H, static_cast<char *>(rows));
    });
    return hipGetLastError();
}

hipError_t launch_combine(const void *rows, const int32_t *slot_pos, const float *weights,
                          int64_t T, int top, int H, int dtype, void *out, hipStream_t stream) {
    by_type(dtype, access(rows, out, nullptr, H, H, dtype), [&](auto d, auto v) {
        constexpr int V = decltype(v)::value, U = unroll<decltype(v)>();
        const dim3 grid((unsigned)T, segments(H, V * U));
        const char *r = static_cast<const char *>(rows);
        char *o = static_cast<char *>(out);
        if (weights)
            combine_kernel<decltype(d)::value, decltype(d)::value, V, U, true><<<grid, kThreads, 0, stream>>>(r, slot_pos, weights, top, T * top, H, o);
        else
            combine_kernel<decltype(d)::value, decltype(d)::value, V, U, false><<<grid, kThreads, 0, stream>>>(r, slot_pos, weights, top, T * top, H, o);
    });
    return hipGetLastError();
}

hipError_t launch_combine_layer(const float *rows, const int32_t *slot_pos, const float *weights,
                                int64_t T, int top, int H, int dtype, void *out, hipStream_t stream) {
    // H is a multiple of 32 and the arrays are aligned: 16 bytes of rows per access
    constexpr int V = 4, U = 2;
    const dim3 grid((unsigned)T, segments(H, V * U));
    const char *r = reinterpret_cast<const char *>(rows);
    char *o = static_cast<char *>(out);
    if (dtype == kBf16)
        combine_kernel<kBf16, kF32, V, U, true><<<grid, kThreads, 0, stream>>>(r, slot_pos, weights, top, T * top, H, o);
    else if (dtype == kF16)
        combine_kernel<kF16, kF32, V, U, true><<<grid, kThreads, 0, stream>>>(r, slot_pos, weights, top, T * top, H, o);
    else
        return launch_combine(rows, slot_pos, weights, T, top, H, dtype, out, stream);
    return hipGetLastError();
}

hipError_t launch_combine_backward(const void *d_out, int64_t ldd, const void *rows,
                                   const int32_t *slot_pos, const float *weights, int64_t T,
                                   int top, int H, int dtype, void *d_rows, float *d_weights,
                                   hipStream_t stream) {
    by_type(dtype, access(d_out, rows, d_rows, ldd, H, dtype), [&](auto d, auto v) {
        combine_backward_kernel<decltype(d)::value, decltype(v)::value><<<dim3((unsigned)T), kThreads, 0, stream>>>(
            static_cast<const char *>(d_out), ldd, static_cast<const char *>(rows), slot_pos, weights,
            top, T * top, H, static_cast<char *>(d_rows), d_weights);
    });
    return hipGetLastError();
}

}  // namespace moe
