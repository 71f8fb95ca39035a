// LDS-tiled 16-bit products with the epilogue fused, for the forward pass and
// both gradients.
//
//   out[m, n] = epilogue( sum_k a(m, k) b(n, k) )
//
// An operand is row-major (k contiguous: x and w of the forward pass, d_pre of
// d_x) or k-major (the rows contiguous: w of d_x, d_pre and x of d_w). No operand
// is transposed in memory: a k-major tile is staged as it lies, 64 rows of k, and
// its fragments are read with gfx950's transposing LDS read
// (ds_read_b64_tr_b16: 16 lanes that address 4 rows of 16 elements receive a
// column of 4 each), so both kinds take the same loads and matrix instructions.
//
//  - A workgroup of GM x GN wavefronts computes a BM x BN tile, each wavefront a
//    part of 16 x 16 tiles of v_mfma_f32_16x16x32 (bf16 or binary16, fp32 accumulators).
//  - Stages of 64 k travel global -> LDS with 16-byte direct-to-LDS loads through two
//    to four buffers, each stage's loads between the MFMAs of the stages before.
//    Row-major tiles: 128-byte rows, chunk c of row r at slot c ^ swz(r). k-major tiles:
//    rows of BM or BN elements, chunk c of row k at slot c ^ kswz(k): the
//    eight rows that half a wavefront reads at once lie in different banks.
//  - Rows past the operand's end are read from its last row (never stored). A last stage of
//    fewer than 64 k is multiplied first, outside the pipeline, with what lies past K masked in
//    the fragments of both operands.
//  - The MFMA takes b first: a lane ends with 4 consecutive outputs of a row. They
//    are staged in fp32 in the wavefront's share of LDS, and bias, activation and
//    residual act on 8 consecutive outputs per lane; the residual is read and the
//    outputs written in whole 16-byte pieces by the same lane (in-place residuals).
//  - With splits > 1, workgroups of one tile take ranges of the stages and leave fp32 partial
//    tiles in a workspace, which join_kernel adds in order and finishes.
//  - Tiles are assigned XCD-contiguously, in groups of 8 tile rows, so that tiles that
//    run at once share operand rows in the same L2.
//
// Measured: 8192 x 8192 x 8192 bf16 1463 TFLOP/s, bound by the card's power (the library's 1602; MFMAs alone on such
// values 1990). 16448 x 5120 x 1280 213 us plain, 244 with gelu and pre: the epilogues of five rounds of
// tiles stand between the products (337 MB of stores). 257 x 1040 x 1312 9.5 us: latency of a stage.
#include <type_traits>

#include "activation.hpp"
#include "launch.hpp"
#include "linear16.hpp"
#include "linear16_mfma.hpp"
#include "quant_math.hpp"
#include "rows.hpp"

namespace linear16 {
namespace {

using rows::kBf16;
using rows::kF16;

constexpr int kStep = 32;      // k of an MFMA
constexpr int kStageK = 64;    // k of a stage: 8 chunks of 16 bytes per row
constexpr int kSteps = kStageK / kStep;

// Slot of chunk c of k row k of a k-major tile of ROWS rows: c ^ kswz(k). Half a wavefront reads
// 32 bytes of k rows 0-3 and 8-11 (from a multiple of 4) at once: 8 distinct 32-byte blocks.
template <int ROWS>
__device__ __forceinline__ int kswz(int k) {
    static_assert(ROWS >= 64, "at least half the banks");
    return ROWS == 64 ? 2 * (((k >> 1) & 1) | ((k >> 2) & 2)) : 2 * ((k & 3) | ((k >> 1) & 4));
}

// A workgroup barrier that waits for all but this wavefront's last N loads and for its LDS
// accesses (see gemm_tiled.hip: no memory fence, loads of later stages stay in flight).
template <int N>
__device__ __forceinline__ void stage_barrier() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (0 << 8) | ((N >> 4) << 14));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The loads of one operand's part of a stage: ROWS rows (of the tile) by 64 k, in 16-byte
// chunks. Load l of wavefront w fills slots 64 (w + WAVES l) ... + 63.
template <bool KM, int ROWS, int WAVES>
struct Loads {
    static constexpr int N = ROWS * 8 / (kWave * WAVES);
    static_assert(N * kWave * WAVES == ROWS * 8, "whole loads");
    const char *p[N];   // this lane's chunk of each load, in the stage to be loaded next
    int64_t step;       // bytes from one stage to the next

    // k_left: k of the first stage, where that is short: chunks past them are read from the last
    // ones (and masked as they are used).
    __device__ __forceinline__ void init(const Operand &o, int64_t r0, int64_t last, int64_t k0, int wave, int lane,
                                         int k_left = kStageK) {
        const char *base = static_cast<const char *>(o.p);
        step = KM ? kStageK * 2 * o.ld : kStageK * 2;
#pragma unroll
        for (int l = 0; l < N; ++l) {
            const int slot = kWave * (wave + WAVES * l) + lane;
            if constexpr (KM) {
                constexpr int per = ROWS / 8;   // chunks of a k row
                const int kr = slot / per, c = (slot % per) ^ kswz<ROWS>(kr);
                p[l] = base + 2 * ((k0 + min(kr, k_left - 1)) * o.ld + min(r0 + 8 * c, last - 7));
            } else {
                const int row = slot / 8, c = (slot % 8) ^ swz(row);
                p[l] = base + 2 * (min(r0 + row, last) * o.ld + k0 + min(8 * c, k_left - 8));
            }
        }
    }
    // Load l of the stage into buf (the operand's slots).
    __device__ __forceinline__ void issue(int l, uint4 *buf, int wave) {
        uint4 *dst = buf + kWave * (wave + WAVES * l);
        __builtin_amdgcn_global_load_lds((global_void *)p[l], (lds_void *)dst, 16, 0, 0);
        p[l] += step;
    }
    __device__ __forceinline__ void issue_all(uint4 *buf, int wave) {
#pragma unroll
        for (int l = 0; l < N; ++l) issue(l, buf, wave);
    }
};

// Fragment reads of one operand: 16 rows (tile i of this wavefront), MFMA step kk of a stage.
template <bool KM, int ROWS, int TILES>
struct Fragments {
    int at[KM ? TILES : 1];   // in bytes (k-major) or 16-byte slots (row-major)
    int group, fswz;

    __device__ __forceinline__ void init(int first, int lane) {
        group = lane >> 4;
        const int i16 = lane & 15;
        if constexpr (KM) {
            const int kr = 8 * group + (i16 >> 2);
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
                const int c = (first + 16 * i) / 8 + ((i16 & 3) >> 1);
                at[i] = (kr * (ROWS / 8) + (c ^ kswz<ROWS>(kr))) * 16 + (i16 & 1) * 8;
            }
            fswz = 0;
        } else {
            at[0] = (first + i16) * 8;
            fswz = swz(i16);
        }
    }
    __device__ __forceinline__ v4i read(const uint4 *buf, int i, int kk) const {
        if constexpr (KM) {
            // (k + 4 and k + 32 have the same swizzle as k)
            const char *p = reinterpret_cast<const char *>(buf) + at[i] + kk * kStep * ROWS * 2;
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)p);
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(p + 4 * ROWS * 2));
            return __builtin_bit_cast(v4i, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            return __builtin_bit_cast(v4i, buf[at[0] + i * 16 * 8 + ((kk * 4 + group) ^ fswz)]);
        }
    }
};

// What a product multiplies. Rows of int8 are taken as 16-bit rows of half their length: their loads,
// LDS slots and fragments are the same bytes, and the MFMA of 64 int8 k takes them as the others take 32.
enum Kind { kKindBf16, kKindF16, kKindInt8 };

template <int KIND, typename A>
__device__ __forceinline__ A multiply_add(v4i a, v4i b, A c) {
    if constexpr (KIND == kKindInt8) return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
    else return mfma<KIND == kKindF16>(a, b, c);
}

struct Tiles {
    Operand a, b;
    int64_t M, N, K;
    int tiles_m, tiles_n;
    int whole;              // tiles of one workgroup each, the first ones in the tile order
    int splits;             // workgroups of each other tile
    float *partial;         // their sums: [tile - whole][split][BM][BN]
    Epilogue ep;
    const float *x_scale, *w_scale;   // int8: of the rows, of the channels
};

// The first row and column of tile t: in groups of 8 tile rows.
__device__ __forceinline__ void tile_at(const Tiles &g, int t, int BM, int BN, int64_t &m0, int64_t &n0) {
    constexpr int kGroup = 8;
    const int per_group = kGroup * g.tiles_n, first_m = t / per_group * kGroup;
    const int gsize = min(g.tiles_m - first_m, kGroup);
    m0 = (int64_t)(first_m + t % per_group % gsize) * BM;
    n0 = (int64_t)(t % per_group / gsize) * BN;
}

// What workgroup `block` computes: the whole tiles, then the parts of the others, each spread over the XCDs
// for themselves.
struct Place {
    bool split;
    int stages, unit, s0, s1;   // of the product; of the parts; the stages of this one
    int64_t m0, n0;

    __device__ __forceinline__ Place(const Tiles &g, int block, int BM, int BN) {
        const int tiles = g.tiles_m * g.tiles_n;
        split = block >= g.whole;
        stages = (int)((g.K + kStageK - 1) / kStageK);
        int t;
        unit = s0 = 0;
        s1 = stages;
        if (split) {
            unit = w8a8::xcd_contiguous(block - g.whole, (tiles - g.whole) * g.splits);
            t = g.whole + unit / g.splits;
            const int part = unit % g.splits;
            s0 = (int)((int64_t)stages * part / g.splits);
            s1 = (int)((int64_t)stages * (part + 1) / g.splits);
        } else {
            t = w8a8::xcd_contiguous(block, g.whole);
        }
        tile_at(g, t, BM, BN, m0, n0);
    }
};

// Eight residual values (0 without a residual), as stored.
__device__ __forceinline__ uint4 residual_at(const Epilogue &ep, int64_t m, int64_t n, bool in) {
    if (!ep.residual || !in) return make_uint4(0, 0, 0, 0);
    return *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(ep.residual) + m * ep.ldr + n);
}

// Outputs (m, n ... n + 7) from their sums.
template <bool F16, bool STREAM>
__device__ __forceinline__ void finish(float (&v)[8], const float (&bias)[8], uint4 residual, const Epilogue &ep, int64_t N,
                                       int64_t m, int64_t n) {
    constexpr auto D = F16 ? kF16 : kBf16;
    auto store = [](void *to, uint4 u) {
        if constexpr (STREAM) w8a8::store16_nt(to, u);
        else *static_cast<uint4 *>(to) = u;
    };
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += bias[e];
    if (ep.pre) store(static_cast<uint16_t *>(ep.pre) + m * N + n, rows::narrow_chunk<D>(v));
    act::activate(ep.act, v);
    if (ep.residual) {
        float r[8];
        rows::widen_chunk<D>(residual, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += r[e];
    }
    store(static_cast<uint16_t *>(ep.out) + m * N + n, rows::narrow_chunk<D>(v));
}

// One K stage: multiply the stage in rd and read the first fragments of the next one from nx.
// The barrier before the last MFMA step says that every wavefront has read all of rd (the last
// step's fragments are in registers by then) and that the next stage has landed; from there on the stage NB
// ahead is loaded into rd, an even share per MFMA step, the last shares beside the next stage's first
// steps: a burst of loads would hold the wavefront's MFMAs. So the first steps here finish the
// loads into `before`, the buffer of the stage before. Fragment reads and loads go out between the
// MFMAs; scheduling barriers pin the order.
struct Ahead {
    bool full;         // the stages that the counted wait assumes are in flight
    bool rest, begin;  // whether there are loads into the buffer before, into this one
};

template <bool F16, int TM, int TN, int BM, int NB, typename LA, typename LB, typename FA, typename FB>
__device__ __forceinline__ void stage(uint4 *__restrict__ rd, const uint4 *__restrict__ nx, uint4 *__restrict__ before, LA &la,
                                      LB &lb, const FA &fa, const FB &fb, const Ahead &h, int wave, v4f (&acc)[TM][TN],
                                      v4i (&xa)[2][TM], v4i (&wb)[2][TN]) {
    constexpr int NLD = LA::N + LB::N, NMF = TM * TN, BSLOT = BM * 8;
    constexpr int LPK = NB == 2 ? NLD : (NLD + kSteps - 1) / kSteps;   // loads per step
    constexpr int GAP = NMF / LPK;                                     // MFMAs per load
    static_assert(GAP >= 1 && kSteps == 2, "a load follows an MFMA; the fragments' two sets alternate");
    constexpr int RPS = (TM + TN + NMF - 1) / NMF;                     // fragment reads per MFMA
#pragma unroll
    for (int kk = 0; kk < kSteps; ++kk) {
        const int f = kk;
        const bool last = kk == kSteps - 1;
        if (last) {
            if (h.full) stage_barrier<(NB - 2) * NLD>();
            else stage_barrier<0>();
        }
        const uint4 *src = last ? nx : rd;
        const int first = last ? 0 : (kk + 1) * LPK;   // of the step's loads
#pragma unroll
        for (int q = 0; q < NMF; ++q) {
            const int i = q / TN, j = q % TN;
            acc[i][j] = mfma<F16>(wb[f][j], xa[f][i], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = 0; r < RPS; ++r) {
                const int x = q * RPS + r;   // a fragment of the next step, in the order of their first use
                if (x == 0) xa[f ^ 1][0] = fa.read(src, 0, (kk + 1) % kSteps);
                else if (x <= TN) wb[f ^ 1][x - 1] = fb.read(src + BSLOT, x - 1, (kk + 1) % kSteps);
                else if (x < TM + TN) xa[f ^ 1][x - TN] = fa.read(src, x - TN, (kk + 1) % kSteps);
            }
            if (q % GAP == GAP - 1 && q / GAP < LPK) {
                const int l = first + q / GAP;
                if (l < NLD && (last ? h.begin : h.rest)) {
                    uint4 *to = last ? rd : before;
                    if (l < LA::N) la.issue(l, to, wave);
                    else lb.issue(l - LA::N, to + BSLOT, wave);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// The words of a fragment with elements past `valid` zeroed.
__device__ __forceinline__ v4i first_elements(v4i f, int valid) {
#pragma unroll
    for (int w = 0; w < 4; ++w) f[w] = 2 * w + 1 < valid ? f[w] : 2 * w < valid ? f[w] & 0xFFFF : 0;
    return f;
}

// The products of a stage of k_left < 64 k, outside the pipeline: what lies past them counts as 0 on both
// sides, whatever was read there.
template <int KIND, int TM, int TN, int BM, typename FA, typename FB, typename A>
__device__ __forceinline__ void short_stage(const uint4 *__restrict__ rd, const FA &fa, const FB &fb, int k_left, int lane,
                                            A (&acc)[TM][TN]) {
#pragma unroll
    for (int kk = 0; kk < kSteps; ++kk) {
        const int valid = k_left - kStep * kk - 8 * (lane >> 4);
        v4i w[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) w[j] = first_elements(fb.read(rd + BM * 8, j, kk), valid);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const v4i x = first_elements(fa.read(rd, i, kk), valid);
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = multiply_add<KIND>(w[j], x, acc[i][j]);
        }
    }
}

// The largest of n, n / 2, n / 4 ... up to most.
constexpr int rows_staged(int n, int most) { return n <= most ? n : rows_staged(n / 2, most); }

// 16-byte slots of a workgroup's stages.
template <int BM, int BN, int NB> constexpr int kSlots = NB * (BM + BN) * 8;

// Workgroup `block` of a product.
template <bool F16, int BM, int BN, int GM, int GN, int NB, bool KA, bool KB, bool TAIL>
__device__ __forceinline__ void tile(const Tiles &g, const int block, uint4 *__restrict__ lds) {
    constexpr int WAVES = GM * GN, WM = BM / GM, WN = BN / GN, TM = WM / 16, TN = WN / 16;
    constexpr int STAGE = (BM + BN) * 8, BSLOT = BM * 8;   // 16-byte slots
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / GN, wn = wave % GN;

    const Place place(g, block, BM, BN);
    const bool split = place.split;
    const int stages = place.stages, unit = place.unit, s0 = place.s0;
    int s1 = place.s1;
    const int64_t m0 = place.m0, n0 = place.n0;

    Fragments<KA, BM, TM> fa;
    Fragments<KB, BN, TN> fb;
    fa.init(wm * WM, lane);
    fb.init(wn * WN, lane);
    v4f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = v4f{};

    Loads<KA, BM, WAVES> la;
    Loads<KB, BN, WAVES> lb;
    constexpr int NLD = la.N + lb.N;
    int at = 0;   // buffer of the first stage
    if (TAIL && s1 == stages) {
        // the product's last, short stage goes first, through buffer 0, while the whole ones arrive
        --s1;
        const int k_left = (int)(g.K - (int64_t)s1 * kStageK);
        la.init(g.a, m0, g.M - 1, (int64_t)s1 * kStageK, wave, lane, k_left);
        lb.init(g.b, n0, g.N - 1, (int64_t)s1 * kStageK, wave, lane, k_left);
        la.issue_all(lds, wave);
        lb.issue_all(lds + BSLOT, wave);
        la.init(g.a, m0, g.M - 1, (int64_t)s0 * kStageK, wave, lane);
        lb.init(g.b, n0, g.N - 1, (int64_t)s0 * kStageK, wave, lane);
#pragma unroll
        for (int b = 1; b < NB; ++b)
            if (s0 + b - 1 < s1) {
                la.issue_all(lds + b * STAGE, wave);
                lb.issue_all(lds + b * STAGE + BSLOT, wave);
            }
        if (s0 + NB - 1 <= s1) stage_barrier<(NB - 1) * NLD>();
        else stage_barrier<0>();
        short_stage<F16, TM, TN, BM>(lds, fa, fb, k_left, lane, acc);
        if (s0 + NB - 1 <= s1) stage_barrier<(NB - 2) * NLD>();
        else stage_barrier<0>();
        if (s0 + NB - 1 < s1) {
            la.issue_all(lds, wave);
            lb.issue_all(lds + BSLOT, wave);
        }
        at = 1;
    } else if (s0 < s1) {
        la.init(g.a, m0, g.M - 1, (int64_t)s0 * kStageK, wave, lane);
        lb.init(g.b, n0, g.N - 1, (int64_t)s0 * kStageK, wave, lane);
#pragma unroll
        for (int b = 0; b < NB; ++b)
            if (s0 + b < s1) {
                la.issue_all(lds + b * STAGE, wave);
                lb.issue_all(lds + b * STAGE + BSLOT, wave);
            }
        if (s0 + NB - 1 < s1) stage_barrier<(NB - 1) * NLD>();
        else stage_barrier<0>();
    }
    if (s0 < s1) {
        v4i xa[2][TM], wb[2][TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) xa[0][i] = fa.read(lds + at * STAGE, i, 0);
#pragma unroll
        for (int j = 0; j < TN; ++j) wb[0][j] = fb.read(lds + at * STAGE + BSLOT, j, 0);
        int before = at == 0 ? NB - 1 : at - 1;
        for (int s = s0; s < s1; ++s) {
            const int next = at == NB - 1 ? 0 : at + 1;
            const Ahead h{s + NB - 1 < s1, s > s0 && s + NB - 1 < s1, s + NB < s1};
            stage<F16, TM, TN, BM, NB>(lds + at * STAGE, lds + next * STAGE, lds + before * STAGE, la, lb, fa, fb, h, wave, acc, xa, wb);
            before = at;
            at = next;
        }
    }
    __syncthreads();

    // tile (i, j), element r of a lane: row 16 i + lane % 16 of the wavefront's part, column
    // 16 j + 4 (lane / 16) + r
    constexpr int kShare = NB * STAGE / WAVES;                       // 16-byte slots
    constexpr int kPass = rows_staged(WM, kShare * 16 / (WN * 4));   // rows staged at a time
    static_assert(kPass >= 16, "passes of whole tiles");
    constexpr int CH = WN / 4, PM = CH - 1;
    static_assert((CH & PM) == 0, "the row-chunk permutation needs a power of two");
    float4 *st = reinterpret_cast<float4 *>(lds) + wave * kShare;
    const int group = lane >> 4, row16 = lane & 15;
    const int lane_n = lane % (WN / 8) * 8;
    const int64_t n = n0 + wn * WN + lane_n;
    float bias[8];
    rows::load_vector<kBf16, true>(g.ep.bias, (int)n, (int)g.N, 0.0f, bias);
#pragma unroll
    for (int p = 0; p < WM / kPass; ++p) {
        if (p) __syncthreads();
#pragma unroll
        for (int i = 0; i < kPass / 16; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int ml = i * 16 + row16;
                st[ml * CH + ((j * 4 + group) ^ (ml & PM))] = __builtin_bit_cast(float4, acc[p * (kPass / 16) + i][j]);
            }
        __syncthreads();
        // kAhead rows' residuals are on their way while as many rows are finished
        constexpr int kTurns = kPass * (WN / 8) / kWave, kAhead = kTurns < 4 ? kTurns : 4;
        static_assert(kTurns % kAhead == 0, "whole groups of turns");
        auto row_of = [&](int it) { return it * (kWave / (WN / 8)) + lane / (WN / 8); };
        auto residual_of = [&](int it) {
            const int64_t m = m0 + wm * WM + p * kPass + row_of(it);
            return residual_at(g.ep, m, n, !split && m < g.M && n < g.N);
        };
        uint4 res[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) res[u] = residual_of(u);
#pragma nounroll
        for (int it0 = 0; it0 < kTurns; it0 += kAhead) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int it = it0 + u, ml = row_of(it), row = wm * WM + p * kPass + ml;
                const uint4 r = res[u];
                if (it + kAhead < kTurns) res[u] = residual_of(it + kAhead);
                if (m0 + row >= g.M || n >= g.N) continue;
                float v[8];
                *reinterpret_cast<float4 *>(v) = st[ml * CH + ((lane_n / 4) ^ (ml & PM))];
                *reinterpret_cast<float4 *>(v + 4) = st[ml * CH + ((lane_n / 4 + 1) ^ (ml & PM))];
                if (split) {
                    float4 *to = reinterpret_cast<float4 *>(g.partial + ((int64_t)unit * BM + row) * BN + wn * WN + lane_n);
                    to[0] = *reinterpret_cast<float4 *>(v);
                    to[1] = *reinterpret_cast<float4 *>(v + 4);
                } else {
                    finish<F16, true>(v, bias, r, g.ep, g.N, m0 + row, n);
                }
            }
        }
    }
}

// The tile of 64 x 64 where few of them leave CUs idle: each of 4 wavefronts takes the whole tile over every
// fourth stage, through two buffers of its own, so no barrier stands in its loop and a stage's chain of load, LDS
// read and MFMA runs four times beside itself (257 x 1040 x 1312, 85 tiles of 21 stages: 10.8 -> 9.6 us; 300 x 2048 x
// 2048 13.3 -> 10.4; with 512 tiles of 64 stages 33.1 against 29.1; int8 256 x 2176 x 8064 26.3 -> 15.9). The four sums
// are added in LDS in order.
constexpr int kDeepWaves = 4, kDeepBuffers = 2, kDeepStage = (64 + 64) * 8, kDeepSlots = kDeepWaves * kDeepBuffers * kDeepStage;

template <int KIND, typename FA, typename FB, typename A>
__device__ __forceinline__ void whole_stage(const uint4 *__restrict__ rd, const FA &fa, const FB &fb, A (&acc)[4][4]) {
    v4i x[kSteps][4], w[kSteps][4];
#pragma unroll
    for (int kk = 0; kk < kSteps; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[kk][i] = fa.read(rd, i, kk);
            w[kk][i] = fb.read(rd + 64 * 8, i, kk);
        }
#pragma unroll
    for (int kk = 0; kk < kSteps; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = multiply_add<KIND>(w[kk][j], x[kk][i], acc[i][j]);
}

// A wavefront's own loads and LDS reads: all but the last N loads have landed; all reads are done.
template <int N>
__device__ __forceinline__ void wait_loads() {
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

template <int KIND, bool KA, bool KB, bool TAIL>
__device__ __forceinline__ void deep_tile(const Tiles &g, const int block, uint4 *__restrict__ lds) {
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const Place place(g, block, 64, 64);
    uint4 *const mine = lds + wave * kDeepBuffers * kDeepStage;

    Fragments<KA, 64, 4> fa;
    Fragments<KB, 64, 4> fb;
    fa.init(0, lane);
    fb.init(0, lane);
    typedef typename std::conditional<KIND == kKindInt8, v4i, v4f>::type Sum;
    Sum acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = Sum{};

    Loads<KA, 64, 1> la;
    Loads<KB, 64, 1> lb;
    constexpr int NLD = la.N + lb.N;
    auto init = [&](int stage, int k_left) {
        la.init(g.a, place.m0, g.M - 1, (int64_t)stage * kStageK, 0, lane, k_left);
        lb.init(g.b, place.n0, g.N - 1, (int64_t)stage * kStageK, 0, lane, k_left);
        la.step *= kDeepWaves;
        lb.step *= kDeepWaves;
    };
    auto issue = [&](int buffer) {
        la.issue_all(mine + buffer * kDeepStage, 0);
        lb.issue_all(mine + buffer * kDeepStage + 64 * 8, 0);
    };
    // the product's last, short stage goes first, to the wavefront whose turn it would be
    const bool tail = TAIL && place.s1 == place.stages;
    const int whole = place.s1 - place.s0 - tail;
    const int count = (whole - wave + kDeepWaves - 1) / kDeepWaves;   // (0 for whole < wave, too)
    int at = 0;   // buffer of the first whole stage
    if (TAIL && tail && whole % kDeepWaves == wave) {
        const int k_left = (int)(g.K - (int64_t)(place.s1 - 1) * kStageK);
        init(place.s1 - 1, k_left);
        issue(0);
        if (count > 0) {
            init(place.s0 + wave, kStageK);
            issue(1);
            wait_loads<NLD>();
        } else {
            wait_loads<0>();
        }
        short_stage<KIND, 4, 4, 64>(mine, fa, fb, k_left, lane, acc);
        wait_reads();
        if (count > 1) issue(0);
        at = 1;
    } else if (count > 0) {
        init(place.s0 + wave, kStageK);
        issue(0);
        if (count > 1) issue(1);
    }
    for (int i = 0; i < count; ++i) {
        if (i + 1 < count) wait_loads<NLD>();
        else wait_loads<0>();
        whole_stage<KIND>(mine + at * kDeepStage, fa, fb, acc);
        wait_reads();   // before its buffer is filled again
        if (i + 2 < count) issue(at);
        at ^= 1;
    }

    // a thread finishes two pieces of 8 outputs
    constexpr int CH = 16, PM = CH - 1;   // 16-byte chunks of a row of sums
    const int row0 = threadIdx.x / 8, col = threadIdx.x % 8 * 8;
    const int64_t n = place.n0 + col;
    float bias[8];
    rows::load_vector<kBf16, true>(g.ep.bias, (int)n, (int)g.N, 0.0f, bias);
    uint4 residual[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t m = place.m0 + row0 + 32 * h;
        residual[h] = residual_at(g.ep, m, n, !place.split && m < g.M && n < g.N);
    }
    float w_scale[8], x_scale[2];
    if constexpr (KIND == kKindInt8) {
        rows::load_vector<kBf16, true>(g.w_scale, (int)n, (int)g.N, 0.0f, w_scale);
#pragma unroll
        for (int h = 0; h < 2; ++h) x_scale[h] = g.x_scale[min(place.m0 + row0 + 32 * h, g.M - 1)];
    }
    Sum *const sums = reinterpret_cast<Sum *>(mine);   // (this wavefront's reads are done)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = 16 * i + (lane & 15);
            sums[row * CH + ((j * 4 + (lane >> 4)) ^ (row & PM))] = acc[i][j];
        }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = row0 + 32 * h;
        const int64_t m = place.m0 + row;
        if (m >= g.M || n >= g.N) continue;
        Sum sum[2];
#pragma unroll
        for (int w = 0; w < kDeepWaves; ++w)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const Sum f = reinterpret_cast<const Sum *>(lds + w * kDeepBuffers * kDeepStage)[row * CH + ((col / 4 + q) ^ (row & PM))];
                sum[q] = w ? sum[q] + f : f;
            }
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (KIND == kKindInt8)
                v[e] = w8a8::dequant(sum[e / 4][e % 4], w8a8::split_scale(x_scale[h]), w8a8::split_scale(w_scale[e]));
            else
                v[e] = sum[e / 4][e % 4];
        }
        if (place.split) {
            float4 *to = reinterpret_cast<float4 *>(g.partial + ((int64_t)place.unit * 64 + row) * 64 + col);
            to[0] = make_float4(v[0], v[1], v[2], v[3]);
            to[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            finish<KIND == kKindF16, true>(v, bias, residual[h], g.ep, g.N, m, n);
        }
    }
}

template <int KIND, bool KA, bool KB, bool TAIL>
__global__ __launch_bounds__(kDeepWaves *kWave, 1) void deep_kernel(const Tiles g) {
    __shared__ uint4 lds[kDeepSlots];
    w8a8::lds_poison(lds);
    w8a8::lds_poison_done();
    deep_tile<KIND, KA, KB, TAIL>(g, blockIdx.x, lds);
}

template <bool F16, int BM, int BN, int GM, int GN, int NB, int OCC, bool KA, bool KB, bool TAIL>
__global__ __launch_bounds__(GM *GN *kWave, GM *GN *OCC / 4) void tiled_kernel(const Tiles g) {
    __shared__ uint4 lds[kSlots<BM, BN, NB>];
    w8a8::lds_poison(lds);
    w8a8::lds_poison_done();
    tile<F16, BM, BN, GM, GN, NB, KA, KB, TAIL>(g, blockIdx.x, lds);
}

// Both gradients in one launch: the workgroups of one fill the chip where those of the other leave it
// idle at their end.
struct Pair {
    Tiles x, w;             // d_x and d_w
    int x_first, w_first;   // their first workgroups
    int w_blocks;
};

template <bool F16, int BM, int BN, int GM, int GN, int NB, int OCC, bool TX, bool TW>
__global__ __launch_bounds__(GM *GN *kWave, GM *GN *OCC / 4) void pair_kernel(const Pair p) {
    __shared__ uint4 lds[kSlots<BM, BN, NB>];
    w8a8::lds_poison(lds);
    w8a8::lds_poison_done();
    const int w = (int)blockIdx.x - p.w_first;
    if (w >= 0 && w < p.w_blocks) tile<F16, BM, BN, GM, GN, NB, true, true, TW>(p.w, w, lds);
    else tile<F16, BM, BN, GM, GN, NB, false, true, TX>(p.x, (int)blockIdx.x - p.x_first, lds);
}

// The sums of the parts of the split tiles and the epilogue: 8 outputs per thread of the first
// slice. SLICES slices of the parts are summed in order, then the slices.
template <bool F16, int BM, int BN, int SLICES>
__global__ __launch_bounds__(256) void join_kernel(const Tiles g) {
    constexpr int kChunks = 256 / SLICES, kBlocks = BM * BN / 8 / kChunks;   // workgroups of a tile
    __shared__ float4 red[SLICES > 1 ? SLICES - 1 : 1][kChunks][2];
    w8a8::lds_poison(red);
    w8a8::lds_poison_done();
    const int i = threadIdx.x % kChunks, slice = threadIdx.x / kChunks;
    const int tile = blockIdx.x / kBlocks, chunk = blockIdx.x % kBlocks * kChunks + i;
    const int row = chunk / (BN / 8), col = chunk % (BN / 8) * 8;
    int64_t m0, n0;
    tile_at(g, g.whole + tile, BM, BN, m0, n0);
    const int64_t m = m0 + row, n = n0 + col;
    const bool in = m < g.M && n < g.N;
    float v[8] = {}, bias[8];
    rows::load_vector<kBf16, true>(slice ? nullptr : g.ep.bias, (int)n, (int)g.N, 0.0f, bias);
    const uint4 residual = residual_at(g.ep, m, n, in && !slice);
    if (in) {
        const float *from = g.partial + ((int64_t)tile * g.splits * BM + row) * BN + col;
#pragma unroll 4
        for (int s = slice; s < g.splits; s += SLICES) {
            const float4 *p = reinterpret_cast<const float4 *>(from + (int64_t)s * (BM * BN));
            const float4 lo = p[0], hi = p[1];
            v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
            v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
        }
    }
    if constexpr (SLICES > 1) {
        if (slice) {
            red[slice - 1][i][0] = make_float4(v[0], v[1], v[2], v[3]);
            red[slice - 1][i][1] = make_float4(v[4], v[5], v[6], v[7]);
        }
        __syncthreads();
        if (slice) return;
#pragma unroll
        for (int s = 0; s < SLICES - 1; ++s) {
            const float4 lo = red[s][i][0], hi = red[s][i][1];
            v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
            v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
        }
    }
    if (in) finish<F16, false>(v, bias, residual, g.ep, g.N, m, n);
}

// Many parts of few tiles are summed in 8 slices.
template <bool F16, int BM, int BN>
hipError_t launch_join(const Tiles &g, int tiles, hipStream_t stream) {
    if (g.splits > 8) join_kernel<F16, BM, BN, 8><<<dim3((unsigned)(tiles * (BM * BN / 8 / 32))), 256, 0, stream>>>(g);
    else join_kernel<F16, BM, BN, 1><<<dim3((unsigned)(tiles * (BM * BN / 8 / 256))), 256, 0, stream>>>(g);
    return hipGetLastError();
}

// Counts a product's tiles; the workgroups that they take.
template <int BM, int BN>
int blocks_of(Tiles &g) {
    g.tiles_m = (int)((g.M + BM - 1) / BM);
    g.tiles_n = (int)((g.N + BN - 1) / BN);
    return g.whole + (g.tiles_m * g.tiles_n - g.whole) * g.splits;
}

template <bool F16, int BM, int BN, int GM, int GN, int NB, int OCC>
hipError_t launch_both(Tiles x, Tiles w, bool w_first, hipStream_t stream) {
    const int nx = blocks_of<BM, BN>(x), nw = blocks_of<BM, BN>(w);
    const Pair p{x, w, w_first ? nw : 0, w_first ? 0 : nx, nw};
    const dim3 grid((unsigned)(nx + nw)), block(GM * GN * kWave);
    const bool tx = x.K % kStageK != 0, tw = w.K % kStageK != 0;
    if (tx && tw) pair_kernel<F16, BM, BN, GM, GN, NB, OCC, true, true><<<grid, block, 0, stream>>>(p);
    else if (tx) pair_kernel<F16, BM, BN, GM, GN, NB, OCC, true, false><<<grid, block, 0, stream>>>(p);
    else if (tw) pair_kernel<F16, BM, BN, GM, GN, NB, OCC, false, true><<<grid, block, 0, stream>>>(p);
    else pair_kernel<F16, BM, BN, GM, GN, NB, OCC, false, false><<<grid, block, 0, stream>>>(p);
    hipError_t e = hipGetLastError();
    for (const Tiles *g : {&x, &w}) {
        const int shared = g->tiles_m * g->tiles_n - g->whole;
        if (e == hipSuccess && shared) e = launch_join<F16, BM, BN>(*g, shared, stream);
    }
    return e;
}

template <bool F16, int BM, int BN, int GM, int GN, int NB, int OCC, bool KA, bool KB>
hipError_t launch(Tiles g, hipStream_t stream) {
    const dim3 grid((unsigned)blocks_of<BM, BN>(g)), block(GM * GN * kWave);
    if (g.K % kStageK == 0) tiled_kernel<F16, BM, BN, GM, GN, NB, OCC, KA, KB, false><<<grid, block, 0, stream>>>(g);
    else tiled_kernel<F16, BM, BN, GM, GN, NB, OCC, KA, KB, true><<<grid, block, 0, stream>>>(g);
    const hipError_t e = hipGetLastError();
    const int shared = g.tiles_m * g.tiles_n - g.whole;
    return e != hipSuccess || !shared ? e : launch_join<F16, BM, BN>(g, shared, stream);
}

template <int KIND, bool KA, bool KB>
hipError_t launch_deep(Tiles g, hipStream_t stream) {
    const dim3 grid((unsigned)blocks_of<64, 64>(g)), block(kDeepWaves * kWave);
    if (g.K % kStageK == 0) deep_kernel<KIND, KA, KB, false><<<grid, block, 0, stream>>>(g);
    else deep_kernel<KIND, KA, KB, true><<<grid, block, 0, stream>>>(g);
    const hipError_t e = hipGetLastError();
    const int shared = g.tiles_m * g.tiles_n - g.whole;
    return e != hipSuccess || !shared ? e : launch_join<KIND == kKindF16, 64, 64>(g, shared, stream);
}

template <bool F16, bool KA, bool KB>
hipError_t launch_form(const Tiles &g, int form, hipStream_t stream) {
    switch (form) {
        case k256x256: return launch<F16, 256, 256, 4, 2, 2, 1, KA, KB>(g, stream);
        case k256x128: return launch<F16, 256, 128, 4, 2, 3, 1, KA, KB>(g, stream);
        case k128x128: return launch<F16, 128, 128, 2, 4, 2, 2, KA, KB>(g, stream);
        case k128x128deep: return launch<F16, 128, 128, 4, 2, 4, 1, KA, KB>(g, stream);
        case k64x64: return launch<F16, 64, 64, 2, 2, 3, 3, KA, KB>(g, stream);
        default: return launch_deep<F16, KA, KB>(g, stream);
    }
}

template <bool F16>
hipError_t launch_pair_form(const Tiles &x, const Tiles &w, int form, bool w_first, hipStream_t stream) {
    switch (form) {
        case k256x256: return launch_both<F16, 256, 256, 4, 2, 2, 1>(x, w, w_first, stream);
        case k128x128: return launch_both<F16, 128, 128, 2, 4, 2, 2>(x, w, w_first, stream);
        default: return launch_both<F16, 64, 64, 2, 2, 3, 3>(x, w, w_first, stream);
    }
}

template <bool F16>
hipError_t launch_type(const Tiles &g, int form, hipStream_t stream) {
    if (g.a.k_major) return launch_form<F16, true, true>(g, form, stream);
    return g.b.k_major ? launch_form<F16, false, true>(g, form, stream) : launch_form<F16, false, false>(g, form, stream);
}

}  // namespace

hipError_t launch_tiled(const Operand &a, const Operand &b, int64_t M, int64_t N, int64_t K, bool f16, const Plan &plan,
                        float *partial, const Epilogue &ep, hipStream_t stream) {
    const Tiles g{a, b, M, N, K, 0, 0, plan.whole, plan.splits, partial, ep, nullptr, nullptr};
    return f16 ? launch_type<true>(g, plan.form, stream) : launch_type<false>(g, plan.form, stream);
}

hipError_t launch_int8(const int8_t *xq, const float *x_scale, int64_t M, const int8_t *wq, const float *w_scale, int64_t N,
                       int64_t K, const Epilogue &ep, hipStream_t stream) {
    const int64_t half = K / 2;
    const int tiles = (int)((M + 63) / 64 * ((N + 63) / 64));
    return launch_deep<kKindInt8, false, false>(Tiles{{xq, half, false}, {wq, half, false}, M, N, half, 0, 0, tiles, 1, nullptr,
                                                      ep, x_scale, w_scale}, stream);
}

hipError_t launch_pair(const Product &x, const Product &w, bool f16, const PairPlan &plan, float *partial,
                       hipStream_t stream) {
    auto tiles = [](const Product &p, const Plan &plan, float *partial) {
        return Tiles{p.a, p.b, p.M, p.N, p.K, 0, 0, plan.whole, plan.splits, partial,
                     Epilogue{nullptr, nullptr, 0, nullptr, p.out, act::kNone}, nullptr, nullptr};
    };
    const Tiles tx = tiles(x, plan.x, partial), tw = tiles(w, plan.w, partial + plan.x.workspace / 4);
    return f16 ? launch_pair_form<true>(tx, tw, plan.x.form, plan.w_first, stream)
               : launch_pair_form<false>(tx, tw, plan.x.form, plan.w_first, stream);
}

}  // namespace linear16
