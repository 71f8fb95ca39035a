// LDS-tiled MXFP4 products (many rows): a dense layer, or rows grouped by
// expert.
//
//   out[m, n] = sum over blocks b of 2^(ex[m,b] + ew[n,b]) * sum_{k in b} qx[m,k] qw[n,k]
//
// A workgroup of GM x GN wavefronts computes a BM x BN tile; each wavefront owns
// a (BM/GM) x (BN/GN) part as 32x32 tiles of v_mfma_scale_f32_32x32x64_f8f6f4,
// which takes two fp4 blocks of 32 per row and their scales and accumulates
// in fp32. A K stage is CH = 8 chunks of 16 bytes per row (256 elements, 8
// scale bytes) or CH = 4 (128 elements, 4 scale bytes). Lanes 0-31 take the
// first half of the stage's blocks and lanes 32-63 the second, for both
// operands, so the stage's K steps use consecutive bytes of one scale register.
//
//  - Codes and scales travel global -> LDS with direct-to-LDS loads (16 and 4
//    bytes per lane) through NB buffers, two stages ahead of the MFMAs. Chunk c
//    of row r sits at slot c ^ swz(r), which keeps the 16-byte fragment reads
//    free of bank conflicts. Scales lie as 32-bit words: CH = 8, one per lane of a
//    32-row fragment; CH = 4, one per row, read by both halves.
//  - Codes of rows past the group or N are not read (they are 0; the scales are
//    the last valid row's), and the outputs are never stored. Blocks past K are
//    read from inside the row; both sides' scale codes there are the storage's
//    padding 0, so that each product is below 2^-240 and adds nothing in fp32.
//  - Rows grouped by expert read their activation row through row_token, so no
//    sorted copy of the activations exists. A wavefront whose rows lie past the
//    group's end only loads.
//  - The MFMA takes the weight first: a lane ends with 4 consecutive channels
//    of a row. Outputs are staged in the wavefront's own LDS and stored as
//    16-byte pieces of contiguous rows; SwiGLU joins gate and up in registers
//    and stores the hidden activations as MXFP4, 17/64 of their bf16 bytes.
//
// What bounds it (8192 x 8192, weights and rows in the Infinity Cache): 34 us for the
// stores (134 MB, 20 us at 6.7 TB/s), the starts and the tiles' ends, and 1.66 us
// (K = 2048 to 4096; 1.78 to 8192, where the clock falls) for each K stage of the 256 x
// 256 tiles: 5.2 PFLOP/s, where the MFMA loop alone reaches 5.7 with one wavefront
// per SIMD and 6.6 with two. A stage's operands alone, two stages under way, take
// 0.71 us (92 GB/s per CU); so the MFMAs, two thirds of a stage's clocks, are what it waits
// for most, and the rest are the barrier and the loads that start behind it. A tile with
// more products per byte is faster until too few tiles are left (tiled_form in
// mxfp4_gemm.hip). 2048 x 4096 x 4096 20-21 us, 38400 x 4096 x 1024 111 us (124
// in a loop of products alone), 32 experts' gate and up of 8192 tokens x 4 310 us, their
// down products to fp32 242 us (199 with the weights in the Infinity Cache; to bf16
// 200 and 179).
#include <algorithm>

#include "launch.hpp"
#include "mxfp4_epilogue.hpp"
#include "mxfp4_form.hpp"

namespace mxfp4 {
namespace {

using w8a8::vm_barrier;

typedef __attribute__((address_space(3))) void lds_void;

// 8 consecutive rows that read the same chunk meet 8 distinct 16-byte bank groups.
template <int CH>
__device__ __forceinline__ int swz(int row) {
    static_assert(CH == 8 || CH == 4, "128- or 64-byte stage rows");
    return CH == 8 ? (row & 7) ^ ((row >> 3) & 1) : ((row >> 1) & 3) ^ ((row >> 3) & 1);
}

struct Operands {
    const uint8_t *xq, *xs, *wq, *ws;
};

// BM x BN outputs by GM x GN wavefronts, CH chunks per row and stage.
template <int BM, int BN, int GM, int GN, int CH>
struct Shape {
    static constexpr int kBM = BM, kBN = BN, kCH = CH, kWaves = GM * GN;
    static constexpr int kBytes = 16 * CH;                        // of codes per row and stage
    static constexpr int kSteps = CH / 2;                         // MFMA K steps per stage
    static constexpr int kRows = 64 / CH;                         // rows per code load of a wavefront
    static constexpr int kA = BM / kRows / kWaves, kB = BN / kRows / kWaves;  // code loads
    // scale loads: rows per load, loads of a wavefront per operand (with fewer
    // loads than wavefronts some repeat another's, so that all wavefronts have
    // the same number of loads in flight)
    static constexpr int kScaleRows = CH == 8 ? 32 : 64;
    static constexpr int kSA = (BM / kScaleRows + kWaves - 1) / kWaves;
    static constexpr int kSB = (BN / kScaleRows + kWaves - 1) / kWaves;
    static constexpr int kLoads = kA + kB + kSA + kSB;
    static constexpr int kCodes = (BM + BN) * CH;                 // 16-byte slots of codes per stage
    static constexpr int kStage = kCodes + (BM + BN) * CH / 16;   // and of scales
};

// Raw buffers and their direct-to-LDS loads of 4 or 16 bytes per lane (types and
// builtins of the device pass; the host pass only parses the kernels).
#ifdef __HIP_DEVICE_COMPILE__
typedef __amdgpu_buffer_rsrc_t Buffer;

// A buffer of `bytes` bytes (at most 2^32 - 1 can be addressed).
__device__ __forceinline__ Buffer buffer(const uint8_t *p, int64_t bytes) {
    const int64_t n = bytes < 0xFFFFFFFFll ? bytes : 0xFFFFFFFFll;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0, (int)(uint32_t)n, 0x00027000);
}

__device__ __forceinline__ void load_lds16(Buffer b, void *dst, uint32_t lane_off, int off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void *)dst, 16, lane_off, off, 0, 0);
}
__device__ __forceinline__ void load_lds4(Buffer b, void *dst, uint32_t lane_off, int off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void *)dst, 4, lane_off, off, 0, 0);
}
#else
struct Buffer {};
__device__ Buffer buffer(const uint8_t *p, int64_t bytes);
__device__ void load_lds16(Buffer b, void *dst, uint32_t lane_off, int off);
__device__ void load_lds4(Buffer b, void *dst, uint32_t lane_off, int off);
#endif

// Codes and scales of activations (a, sa) and weights (b, sb).
struct Sources {
    Buffer a, b, sa, sb;
};

// Where this lane's share of every stage comes from: a buffer per operand, a
// 32-bit offset per lane that stays, and a uniform offset that moves with the
// stage. (Addresses in vector registers cost a 64-bit addition per load, which
// holds up the MFMAs' issue.)
template <typename Sh>
struct Loads {
    Sources src, none;                // none: the same buffers with no bytes (loads give 0)
    int sa_step, sb_step;             // bytes from one 256-element step's scales to the next
    uint32_t aoff[Sh::kA], boff[Sh::kB], saoff[Sh::kSA], sboff[Sh::kSB];
    int kc;                           // chunk of the row that this lane loads
    int half_k;                       // bytes of a row
    int nk;                           // stages

    __device__ __forceinline__ Sources at(int j) const { return j < nk ? src : none; }
};

// Load l of stage j: this lane's 16 bytes of codes or 4 bytes of scales.
template <typename Sh, bool KTAIL>
__device__ __forceinline__ void load_one(const Loads<Sh> &g, const Sources &src, int l, int j, uint4 *st,
                                         int wave) {
    constexpr int BM = Sh::kBM, BN = Sh::kBN, CH = Sh::kCH, kWaves = Sh::kWaves;
    if (l < Sh::kA + Sh::kB) {
        uint4 *dst = st + 64 * (wave + kWaves * (l < Sh::kA ? l : l - Sh::kA)) + (l < Sh::kA ? 0 : BM * CH);
        uint32_t off = l < Sh::kA ? g.aoff[l] : g.boff[l - Sh::kA];
        // a chunk past K: the stage's first one instead (it is inside the row)
        if (KTAIL && g.kc * 16 + j * Sh::kBytes >= g.half_k) off -= g.kc * 16;
        load_lds16(l < Sh::kA ? src.a : src.b, dst, off, j * Sh::kBytes);
    } else {
        const int q = l - Sh::kA - Sh::kB;
        const bool is_a = q < Sh::kSA;
        constexpr int kFragsA = BM / Sh::kScaleRows, kFragsB = BN / Sh::kScaleRows;
        const int f = is_a ? (wave + kWaves * q) % kFragsA : kFragsA + (wave + kWaves * (q - Sh::kSA)) % kFragsB;
        uint32_t *dst = reinterpret_cast<uint32_t *>(st + Sh::kCodes) + 64 * f;
        const int step = CH == 8 ? j : j >> 1, word = CH == 8 ? 0 : 4 * (j & 1);
        if (is_a) load_lds4(src.sa, dst, g.saoff[q], step * g.sa_step + word);
        else load_lds4(src.sb, dst, g.sboff[q - Sh::kSA], step * g.sb_step + word);
    }
}

// What a lane holds of a stage: fragments by K step parity, and scales.
template <int TM, int TN>
struct Frags {
    v4i x[2][TM], w[2][TN];
    uint32_t sx[TM], sw[TN];
};

// This lane's scale bytes, in order from byte 0: a word holds them all (CH = 8)
// or those of both halves (CH = 4).
template <int CH>
__device__ __forceinline__ uint32_t lane_scales(uint32_t word, int half) {
    return CH == 8 ? word : word >> (16 * half);
}

// One K stage: multiply the stage held in `rd`, read the first fragments of the
// next stage from `nx`, and load stage s + 2 into `wr`. The barrier before the
// last K step says that every wavefront has read all of this stage's fragments
// and that the next stage has landed. With two buffers `wr` is `rd` again, so
// the loads follow the barrier; with three it is the buffer of the stage
// before, free since the last barrier, so the loads are spread over all K steps
// (256 x 128 tiles, 2048 x 4096 x 4096: 22.9 us in one burst, 19.7 spread). One
// fragment read or load follows an MFMA; the order is pinned, as bursts hold the
// MFMAs. The code is one straight line, the same for every stage (past the last
// one, the loads come from buffers of no bytes and the fragments are not used):
// the compiler moves these MFMAs across branches, down to where their sums are
// used, and then keeps every fragment alive.
template <typename Sh, int NB, bool KTAIL, int TM, int TN>
__device__ __forceinline__ void stage(const Loads<Sh> &g, const uint4 *rd, const uint4 *nx, uint4 *wr,
                                      int s, int wave, int a_frag, int b_frag, int a_scale, int b_scale,
                                      int half, int fswz, v16f (&acc)[TM][TN], Frags<TM, TN> &f) {
    constexpr int CH = Sh::kCH, kSteps = Sh::kSteps;
    constexpr int NMF = TM * TN;
    constexpr int RPS = (TM + TN + NMF - 1) / NMF;                 // reads per MFMA
    constexpr int LSTEP0 = NB == 2 ? kSteps - 1 : 0;               // first K step with loads
    constexpr int LPK = (Sh::kLoads + kSteps - LSTEP0 - 1) / (kSteps - LSTEP0);  // loads per K step
    constexpr int LPRE = NB == 2 ? 0 : (kSteps - 1) * LPK < Sh::kLoads ? (kSteps - 1) * LPK : Sh::kLoads;
    // loads follow the last MFMAs of a K step, where no reads are left
    constexpr int LPS = NMF > 2 ? (LPK + NMF - 3) / (NMF - 2) : LPK;  // loads per MFMA
    constexpr int LFIRST = NMF - (LPK + LPS - 1) / LPS;
    constexpr int kSc = CH == 8 ? 64 : 32;                         // scale words per 32-row fragment
    const Sources src_bufs = g.at(s + 2);
    uint32_t sx[TM], sw[TN];
#pragma unroll
    for (int kk = 0; kk < kSteps; ++kk) {
        const int p = kk & 1;
        const bool last_step = kk == kSteps - 1;
        if (last_step) vm_barrier<LPRE>();  // the loads of this stage may be in flight
        const uint4 *src = last_step ? nx : rd;
        const int ch = (kSteps * half + (kk + 1) % kSteps) ^ fswz;
#pragma unroll
        for (int q = 0; q < NMF; ++q) {
            const int i = q / TN, j = q % TN;
            acc[i][j] = mfma_32x32x64(kk, f.w[p][j], f.sw[j], f.x[p][i], f.sx[i], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = q * RPS; r < (q + 1) * RPS && r < TM + TN; ++r) {
                if (r < TM) f.x[p ^ 1][r] = __builtin_bit_cast(v4i, src[a_frag + r * 32 * CH + ch]);
                else f.w[p ^ 1][r - TM] = __builtin_bit_cast(v4i, src[b_frag + (r - TM) * 32 * CH + ch]);
                if (last_step) {
                    const uint32_t *sc = reinterpret_cast<const uint32_t *>(nx + Sh::kCodes);
                    if (r < TM) sx[r] = lane_scales<CH>(sc[a_scale + kSc * r], half);
                    else sw[r - TM] = lane_scales<CH>(sc[b_scale + kSc * (r - TM)], half);
                }
            }
            if (kk >= LSTEP0 && q >= LFIRST) {
#pragma unroll
                for (int u = (q - LFIRST) * LPS; u < (q - LFIRST + 1) * LPS && u < LPK; ++u) {
                    const int l = (kk - LSTEP0) * LPK + u;
                    if (l < Sh::kLoads) load_one<Sh, KTAIL>(g, src_bufs, l, s + 2, wr, wave);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) f.sx[i] = sx[i];
#pragma unroll
    for (int j = 0; j < TN; ++j) f.sw[j] = sw[j];
}

// Where one tile's operands are: the loads' addresses for this lane.
template <typename Sh>
__device__ __forceinline__ void aim(Loads<Sh> &g, const Operands &op, const Groups &grp,
                                    const Tile &tile, int n0, int N, int K, int KB, int lane, int wave) {
    constexpr int CH = Sh::kCH, kWaves = Sh::kWaves;
    asm volatile("" : "+v"(lane));  // or a persistent kernel keeps the row numbers in registers
    const int lrow = Sh::kRows * wave + lane / CH;
    g.kc = (lane % CH) ^ swz<CH>(lrow);
    g.half_k = K / 2;
    g.nk = (K / 2 + Sh::kBytes - 1) / Sh::kBytes;
    const int rows = tile.m1 - tile.m0;
    // without row_token the tile's own rows, else rows anywhere in xq
    const int64_t row0 = grp.row_token ? 0 : tile.m0;
    const int64_t half_k = K / 2, first_n = (int64_t)tile.e * N + n0;
    const uint8_t *a = op.xq + row0 * half_k, *b = op.wq + first_n * half_k, *sa = op.xs + row0 * 8,
                  *sb = op.ws + ((int64_t)tile.e * KB * N + n0) * 8;
    // codes of rows past the group's or the weight's end are past these ends: no memory is read
    g.src = Sources{buffer(a, (grp.row_token ? grp.T : rows) * half_k), buffer(b, (N - n0) * half_k),
                    buffer(sa, ((int64_t)KB * grp.T - row0) * 8), buffer(sb, ((int64_t)KB * N - n0) * 8)};
    g.none = Sources{buffer(a, 0), buffer(b, 0), buffer(sa, 0), buffer(sb, 0)};
    g.sa_step = grp.T * 8;
    g.sb_step = N * 8;
    constexpr int kPass = Sh::kRows * kWaves;  // rows from one code load to the next
    // scale words: CH = 8, lane l of a fragment: row l % 32, word l / 32; CH = 4, row l
    const int srow = CH == 8 ? lane & 31 : lane, sword = CH == 8 ? 4 * (lane >> 5) : 0;
    auto scale_row = [&](int q, int side, int end) {
        return min((wave + kWaves * q) % (side / Sh::kScaleRows) * Sh::kScaleRows + srow, end - 1);
    };
    int a_row[Sh::kA], s_row[Sh::kSA];
#pragma unroll
    for (int l = 0; l < Sh::kA; ++l) a_row[l] = lrow + kPass * l;
#pragma unroll
    for (int q = 0; q < Sh::kSA; ++q) s_row[q] = scale_row(q, Sh::kBM, rows);
    if (grp.row_token) {
        int token[Sh::kA + Sh::kSA];
#pragma unroll
        for (int l = 0; l < Sh::kA; ++l) token[l] = tile.m0 + min(a_row[l], rows - 1);
#pragma unroll
        for (int q = 0; q < Sh::kSA; ++q) token[Sh::kA + q] = tile.m0 + s_row[q];
        source_rows(grp, token);
#pragma unroll
        for (int l = 0; l < Sh::kA; ++l) a_row[l] = a_row[l] < rows ? token[l] : grp.T;
#pragma unroll
        for (int q = 0; q < Sh::kSA; ++q) s_row[q] = token[Sh::kA + q];
    }
#pragma unroll
    for (int l = 0; l < Sh::kA; ++l) g.aoff[l] = (uint32_t)a_row[l] * (uint32_t)(K / 2) + g.kc * 16;
#pragma unroll
    for (int l = 0; l < Sh::kB; ++l) g.boff[l] = (uint32_t)(lrow + kPass * l) * (uint32_t)(K / 2) + g.kc * 16;
#pragma unroll
    for (int q = 0; q < Sh::kSA; ++q) g.saoff[q] = (uint32_t)s_row[q] * 8 + sword;
#pragma unroll
    for (int q = 0; q < Sh::kSB; ++q) g.sboff[q] = (uint32_t)scale_row(q, Sh::kBN, N - n0) * 8 + sword;
}

template <typename Sh, bool KTAIL>
__device__ __forceinline__ void load_stage(const Loads<Sh> &g, int j, uint4 *st, int wave) {
    const Sources src = g.at(j);
    // the weight's first: the activations' addresses may still be on their way
    constexpr int kA = Sh::kA, kW = Sh::kA + Sh::kB, kSA = kW + Sh::kSA;
#pragma unroll
    for (int l = kA; l < kW; ++l) load_one<Sh, KTAIL>(g, src, l, j, st, wave);
#pragma unroll
    for (int l = kSA; l < Sh::kLoads; ++l) load_one<Sh, KTAIL>(g, src, l, j, st, wave);
#pragma unroll
    for (int l = 0; l < kA; ++l) load_one<Sh, KTAIL>(g, src, l, j, st, wave);
#pragma unroll
    for (int l = kW; l < kSA; ++l) load_one<Sh, KTAIL>(g, src, l, j, st, wave);
}

// Waits for this wavefront's vector-memory operations (vmcnt 0 only).
__device__ __forceinline__ void wait_loads() {
    __builtin_amdgcn_s_waitcnt(0 | (7 << 4) | (15 << 8));
    asm volatile("" ::: "memory");
}

// The wavefront's outputs: piece by piece (32 rows of at most 128 bytes) through
// its own 4 KB of LDS, 16-byte chunks permuted by the low row bits, so that each
// store instruction writes 8 whole cache lines. (Stores straight from the
// accumulators, 32 bytes of a row each: 38400 x 4096 x 1024 118 -> 168 us.)
constexpr int kPieceSlots = 32 * 8;

template <Epilogue EP, int TM, int TN>
__device__ __forceinline__ void store_plain(const v16f (&acc)[TM][TN], uint4 *mine, void *out, int m0,
                                            int m_end, int nw0, int N, int lane) {
    constexpr int SIZE = EP == kOutF32 ? 4 : 2;
    constexpr int PJ = SIZE == 4 || TN == 1 ? 1 : 2;    // 32-channel tiles per piece
    static_assert(TN % PJ == 0, "whole pieces");
    constexpr int CH = PJ * 32 * SIZE / 16;             // 16-byte chunks per row of a piece
    const int row = lane & 31, half = lane >> 5;
    uint4 *mr = mine + row * CH;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; j += PJ) {
#pragma unroll
            for (int p = 0; p < PJ; ++p)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const v16f &a = acc[i][j + p];
                    const float a0 = a[4 * g], a1 = a[4 * g + 1], a2 = a[4 * g + 2], a3 = a[4 * g + 3];
                    if constexpr (EP == kOutF32) {
                        mr[(p * 8 + 2 * g + half) ^ (row & (CH - 1))] = __builtin_bit_cast(uint4, v4f{a0, a1, a2, a3});
                    } else {
                        const uint2 w = EP == kOutBf16
                            ? make_uint2(w8a8::pack_bf16x2(a0, a1), w8a8::pack_bf16x2(a2, a3))
                            : make_uint2(pack_f16x2(a0, a1), pack_f16x2(a2, a3));
                        reinterpret_cast<uint2 *>(mr + ((p * 4 + g) ^ (row & (CH - 1))))[half] = w;
                    }
                }
#pragma unroll
            for (int it = 0; it < 32 * CH / kWave; ++it) {
                const int q = it * kWave + lane, r = q / CH, c = q % CH;
                const int m = m0 + 32 * i + r, n = nw0 + 32 * j + c * (16 / SIZE);
                const uint4 v = mine[r * CH + (c ^ (r & (CH - 1)))];
                if (m < m_end && n < N)
                    w8a8::store16_nt(static_cast<char *>(out) + ((int64_t)m * N + n) * SIZE, v);
            }
        }
}

// One tile per workgroup, or (PERSIST: SwiGLU, whose stores are few) every
// gridDim.x-th: then the first stages of the next tile are on their way before
// the epilogue of a tile. Plain outputs gain nothing from it, as a workgroup
// would wait for its stores with the next tile's loads (38400 x 4096 x 1024:
// 118 us a workgroup per tile, 127 persistent); SwiGLU does (32 experts' gate and
// up of 8192 tokens: 348 -> 335 us).
template <int BM, int BN, int GM, int GN, int CH, int NB, int OCC, bool KTAIL, Epilogue EP>
__global__ __launch_bounds__(GM *GN *kWave, OCC *GM *GN / 4) void tiled_kernel(
    Operands op, Groups grp, int N, int K, int KB, int tiles_m, int tiles_n, int slots, Output o) {
    using Sh = Shape<BM, BN, GM, GN, CH>;
    constexpr bool PERSIST = EP == kSwiglu;
    constexpr int WM = BM / GM, WN = BN / GN, TM = WM / 32, TN = WN / 32;
    // one array per buffer: the compiler then knows that loads into one do not concern
    // reads of the other
    static_assert(NB == 2 || NB == 3, "two or three buffers");
    static_assert(Sh::kWaves * kPieceSlots <= Sh::kStage, "the staged outputs fit a buffer");
    __shared__ uint4 b0[Sh::kStage], b1[Sh::kStage], b2[NB == 3 ? Sh::kStage : 1];
    w8a8::lds_poison(b0);
    w8a8::lds_poison(b1);
    w8a8::lds_poison(b2);
    w8a8::lds_poison_done();

    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / GN, wn = wave % GN;
    const int frag_row = lane & 31, half = lane >> 5;
    const int a_frag = (wm * WM + frag_row) * CH;
    const int b_frag = BM * CH + (wn * WN + frag_row) * CH;
    constexpr int kSc = CH == 8 ? 64 : 32;  // scale words per 32-row fragment
    const int sl = CH == 8 ? lane : frag_row;
    const int a_scale = wm * (WM / 32) * kSc + sl, b_scale = (BM / 32 + wn * (WN / 32)) * kSc + sl;
    const int fswz = swz<CH>(frag_row);

    GroupScan scan{};
    if (grp.offsets) {
        scan = scan_groups<BM>(grp, 0);
        tiles_m = count_tiles<BM>(grp, scan);
    }
    const int tiles = tiles_m * tiles_n;
    // Tiles XCD by XCD, a group's tiles after another's, in parts of up to kPart
    // tile rows by all columns: the tiles that run at once share activation and
    // weight rows in one L2 (a layer of 8192 tokens and 32 experts 609 us with parts
    // of 4 rows that cross groups, 589 so; gate and up read 925 and 632 MB).
    auto locate = [&](const GroupScan &scan, int pid, int &n0) {
        constexpr int kPart = 6;
        const int t = w8a8::xcd_contiguous(pid, tiles);
        const Group own = find_group<BM>(grp, scan, t / tiles_n);
        const int rows = (own.n + BM - 1) / BM, parts = (rows + kPart - 1) / kPart;
        const int per_part = (rows + parts - 1) / parts, in_group = t - own.first * tiles_n;
        const int m = in_group / (per_part * tiles_n) * per_part, in_part = in_group % (per_part * tiles_n);
        const int part = min(rows - m, per_part);
        n0 = in_part / part * BN;
        return Tile{own.e, own.lo + (m + in_part % part) * BM, own.lo + own.n};
    };
    int pid = blockIdx.x;
    if (pid >= tiles) return;
    // Several tiles per CU of the same length: without this all CUs compute, then
    // all store (57-75 GB/s for a CU among few, 21 when all store). The first
    // workgroups start up to 8 us apart within an XCD, the later ones follow them
    // (us: 8192 x 8192, K = 512 47.0 -> 41.4, 2048 89.6 -> 84.1, 4096 145 -> 139; 32
    // experts' down products of 8192 tokens 197 -> 186). SwiGLU's stores are few.
    if (!PERSIST && pid < slots && tiles > 2 * slots)
        for (int wait = pid / 8 % 32; wait > 0; --wait) __builtin_amdgcn_s_sleep(8);
    int n0;
    Tile tile = locate(scan, pid, n0);
    Loads<Sh> g;
    int first = 0;  // buffer of the first stage
    auto start = [&] {
        if (tile.e < 0 || tile.e >= grp.E) return;
        aim(g, op, grp, tile, n0, N, K, KB, lane, wave);
        // the last stage is always in the last buffer: the first one is where
        // the number of stages asks for
        first = g.nk % NB;
        if (first == 0) first = NB;
        first = NB - first;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int at = (first + j) % NB;
            load_stage<Sh, KTAIL>(g, j, at == 0 ? b0 : at == 1 ? b1 : b2, wave);
        }
    };
    start();
    w8a8::vm_barrier<Sh::kLoads>();  // the first stage has landed everywhere
    while (true) {
        v16f acc[TM][TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = v16f{};
        if (tile.e < 0 || tile.e >= grp.E) {
        } else if (tile.m0 + wm * WM >= tile.m1) {
            // no rows for this wavefront: its share of the loads, and the barriers
            for (int s = 0; s < g.nk; ++s) {
                const int at = (first + s + 2) % NB;
                uint4 *wr = at == 0 ? b0 : at == 1 ? b1 : b2;
                if constexpr (NB == 3) load_stage<Sh, KTAIL>(g, s + 2, wr, wave);
                vm_barrier<NB == 3 ? Sh::kLoads : 0>();
                if constexpr (NB == 2) load_stage<Sh, KTAIL>(g, s + 2, wr, wave);
            }
        } else {
            Frags<TM, TN> f;
            const int ch = (Sh::kSteps * half) ^ fswz;
            const uint4 *b = first == 0 ? b0 : first == 1 ? b1 : b2;
            const uint32_t *sc = reinterpret_cast<const uint32_t *>(b + Sh::kCodes);
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                f.x[0][i] = __builtin_bit_cast(v4i, b[a_frag + i * 32 * CH + ch]);
                f.sx[i] = lane_scales<CH>(sc[a_scale + kSc * i], half);
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                f.w[0][j] = __builtin_bit_cast(v4i, b[b_frag + j * 32 * CH + ch]);
                f.sw[j] = lane_scales<CH>(sc[b_scale + kSc * j], half);
            }
#define MXFP4_STAGE(RD, NX, WR, S)                                                                \
    stage<Sh, NB, KTAIL>(g, RD, NX, WR, S, wave, a_frag, b_frag, a_scale, b_scale, half, fswz, acc, f)
            int s = 0;
            if constexpr (NB == 2) {
                if (first == 1) { MXFP4_STAGE(b1, b0, b1, s); ++s; }
                for (; s < g.nk; s += 2) {
                    MXFP4_STAGE(b0, b1, b0, s);
                    MXFP4_STAGE(b1, b0, b1, s + 1);
                }
            } else {
                if (first == 1) { MXFP4_STAGE(b1, b2, b0, s); ++s; }
                if (first != 0) { MXFP4_STAGE(b2, b0, b1, s); ++s; }
                for (; s < g.nk; s += 3) {
                    MXFP4_STAGE(b0, b1, b2, s);
                    MXFP4_STAGE(b1, b2, b0, s + 1);
                    MXFP4_STAGE(b2, b0, b1, s + 2);
                }
            }
#undef MXFP4_STAGE
        }
        const Tile done = tile;
        const int mw0 = done.m0 + wm * WM, nw0 = n0 + wn * WN;
        pid += gridDim.x;
        const bool more = PERSIST && pid < tiles;
        // all fragment reads done, and (empty) loads landed: the buffers are free
        vm_barrier<0>();
        if (more) {
            // (scanned again: kept, it would cost three registers)
            tile = locate(grp.offsets ? scan_groups<BM>(grp, 0) : GroupScan{}, pid, n0);
            start();
        }
        if (done.e >= 0) {
            if constexpr (EP == kSwiglu) {
                Hidden h[TM][TN / 2];
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; j += 2) h[i][j / 2] = quantize_swiglu(acc[i][j], acc[i][j + 1], half);
                // the next tile's loads have landed before any store is under
                // way, so that nothing later waits for the stores with them
                wait_loads();
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; j += 2) {
                        const int m = mw0 + i * 32 + frag_row;
                        store_hidden(h[i][j / 2], o, m, m < done.m1, nw0 + 32 * j, half, N, grp.S);
                    }
            } else {
                store_plain<EP, TM, TN>(acc, b0 + wave * kPieceSlots, o.out, mw0, done.m1, nw0, N, lane);
            }
        } else {
            wait_loads();
        }
        if (!more) break;
        w8a8::lds_barrier();  // every wavefront has waited for its loads
    }
}

template <int BM, int BN, int GM, int GN, int CH, int NB, int OCC, Epilogue EP>
hipError_t launch_epilogue(const Operands &op, const Groups &g, int N, int K, const Output &o,
                           hipStream_t stream) {
    const int KB = (K + kStep - 1) / kStep;
    const int tiles_n = (N + BN - 1) / BN;
    const int64_t tiles_m = most_tiles(g.S, g.E, BM, g.offsets != nullptr);
    const int slots = OCC * w8a8::device_cu_count();  // workgroups that run at once
    const dim3 grid((unsigned)(EP == kSwiglu ? std::min<int64_t>(tiles_m * tiles_n, slots) : tiles_m * tiles_n)), block(GM * GN * kWave);
    if (K % (32 * CH) == 0)
        tiled_kernel<BM, BN, GM, GN, CH, NB, OCC, false, EP><<<grid, block, 0, stream>>>(op, g, N, K, KB, (int)tiles_m, tiles_n, slots, o);
    else
        tiled_kernel<BM, BN, GM, GN, CH, NB, OCC, true, EP><<<grid, block, 0, stream>>>(op, g, N, K, KB, (int)tiles_m, tiles_n, slots, o);
    return hipGetLastError();
}

template <int BM, int BN, int GM, int GN, int CH, int NB, int OCC>
hipError_t launch_plain(const Operands &op, const Groups &g, int N, int K, int epilogue,
                        const Output &o, hipStream_t stream) {
    switch (epilogue) {
        case kOutBf16: return launch_epilogue<BM, BN, GM, GN, CH, NB, OCC, kOutBf16>(op, g, N, K, o, stream);
        case kOutF16: return launch_epilogue<BM, BN, GM, GN, CH, NB, OCC, kOutF16>(op, g, N, K, o, stream);
        default: return launch_epilogue<BM, BN, GM, GN, CH, NB, OCC, kOutF32>(op, g, N, K, o, stream);
    }
}

template <int BM, int BN, int GM, int GN, int CH, int NB, int OCC>
hipError_t launch_shape(const Operands &op, const Groups &g, int N, int K, int epilogue,
                        const Output &o, hipStream_t stream) {
    static_assert(BN / GN >= 64, "a wavefront's channels hold whole blocks of hidden units");
    if (epilogue == kSwiglu)
        return launch_epilogue<BM, BN, GM, GN, CH, NB, OCC, kSwiglu>(op, g, N, K, o, stream);
    return launch_plain<BM, BN, GM, GN, CH, NB, OCC>(op, g, N, K, epilogue, o, stream);
}

}  // namespace

hipError_t launch_gemm_tiled(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq,
                             const uint8_t *ws, const Groups &g, int N, int K, int epilogue,
                             const Output &o, const Form &f, hipStream_t stream) {
    const Operands op{xq, xs, wq, ws};
    if (f.channels == 64) return launch_plain<64, 64, 2, 2, 8, 3, 2>(op, g, N, K, epilogue, o, stream);
    if (f.rows == 64) return launch_shape<64, 128, 2, 2, 8, 3, 2>(op, g, N, K, epilogue, o, stream);
    if (f.rows == 128) return launch_shape<128, 128, 4, 2, 8, 3, 1>(op, g, N, K, epilogue, o, stream);
    if (f.channels == 256) return launch_shape<256, 256, 2, 4, 8, 2, 1>(op, g, N, K, epilogue, o, stream);
    if (f.waves == 8) return launch_shape<256, 128, 4, 2, 8, 3, 1>(op, g, N, K, epilogue, o, stream);
    return launch_shape<256, 128, 2, 2, 4, 3, 2>(op, g, N, K, epilogue, o, stream);
}

}  // namespace mxfp4
