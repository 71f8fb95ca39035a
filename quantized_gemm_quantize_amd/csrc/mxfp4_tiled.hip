// LDS-tiled MXFP4 products (many rows): a dense layer, or rows grouped by
// expert.
//
//   out[m, n] = sum over blocks b of 2^(ex[m,b] + ew[n,b]) * sum_{k in b} qx[m,k] qw[n,k]
//
// A workgroup of 4 wavefronts computes a BM x BN tile; each wavefront owns a
// (BM/2) x (BN/2) part as 32x32 tiles of v_mfma_scale_f32_32x32x64_f8f6f4,
// which takes two fp4 blocks of 32 per row and their scales and accumulates
// in fp32. A K stage is 256 elements: 128 bytes of codes and 8 scale bytes per
// row. Lanes 0-31 take blocks 0-3 of the stage and lanes 32-63 blocks 4-7, for
// both operands, so the stage's four K steps use the four bytes of one scale
// register.
//
//  - Codes and scales travel global -> LDS with direct-to-LDS loads (16 and 4
//    bytes per lane) through a ring of STAGES buffers, loads running STAGES-1
//    stages ahead of the MFMAs. Rows of codes are 128 bytes; chunk c of row r
//    sits at slot c ^ (r % 8) ^ ((r / 8) % 2), which keeps the 16-byte fragment
//    reads free of bank conflicts. Scales lie as one 32-bit word per lane of a
//    32-row fragment.
//  - Rows past the group or N are read from the last valid row (their outputs
//    are never stored). Blocks past K are read from inside the row; both sides'
//    scale codes there are the storage's padding 0, so that each product is
//    below 2^-240 and adds nothing in fp32.
//  - Rows grouped by expert read their activation row through row_token, so no
//    sorted copy of the activations exists.
//  - The MFMA takes the weight first: a lane ends with 4 consecutive channels
//    of a row. Outputs are staged in the wavefront's own LDS and stored as
//    16-byte pieces of contiguous rows; SwiGLU joins gate and up in registers
//    and stores the hidden activations as MXFP4, 17/64 of their bf16 bytes.
#include "launch.hpp"
#include "mxfp4_epilogue.hpp"

namespace mxfp4 {
namespace {

using w8a8::vm_barrier;

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kChunks = 8;    // 16-byte chunks of codes per row and stage
constexpr int kSteps = 4;     // MFMA K steps per stage

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) void global_void;

__device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }

struct Operands {
    const uint8_t *xq, *xs, *wq, *ws;
};

template <int BM, int BN>
struct Shape {
    static constexpr int kA = BM / 32, kB = BN / 32;              // code loads per wavefront and stage
    static constexpr int kScale = (BM + BN) / 32 / kWaves;        // scale loads per wavefront and stage
    static constexpr int kLoads = kA + kB + kScale;
    static constexpr int kCodes = (BM + BN) * kChunks;            // 16-byte slots of codes per stage
    static constexpr int kStage = kCodes + (BM + BN) / 2;         // and of scales
};

// Where this lane's share of every stage comes from, and what it fills: a
// uniform address that moves with the stage, plus a 32-bit offset per lane that
// does not (64-bit addresses per lane would not fit the registers).
template <int BM, int BN>
struct Loads {
    using Sh = Shape<BM, BN>;
    const uint8_t *a, *b, *sa, *sb;   // uniform
    int64_t sa_step, sb_step;         // bytes from one stage's scales to the next
    uint32_t aoff[Sh::kA], boff[Sh::kB], soff[Sh::kScale];
    int kc;                           // chunk of the row that this lane loads
    int half_k;                       // bytes of a row
    int nk;                           // stages
};

// Load l of stage j: this lane's 16 bytes of codes or 4 bytes of scales.
template <int BM, int BN, bool KTAIL>
__device__ __forceinline__ void load_one(const Loads<BM, BN> &g, int l, int j, uint4 *st, int wave) {
    using Sh = Shape<BM, BN>;
    static_assert(BM / 32 % kWaves == 0, "a scale load is of one operand in every wavefront");
    if (l < Sh::kA + Sh::kB) {
        uint4 *dst = st + 64 * wave + (l < Sh::kA ? 256 * l : BM * kChunks + 256 * (l - Sh::kA));
        const uint8_t *base = (l < Sh::kA ? g.a : g.b) + (int64_t)j * kStepBytes;
        uint32_t off = l < Sh::kA ? g.aoff[l] : g.boff[l - Sh::kA];
        // a chunk past K: the stage's first one instead (it is inside the row)
        if (KTAIL && g.kc * 16 + j * kStepBytes >= g.half_k) off -= g.kc * 16;
        __builtin_amdgcn_global_load_lds((global_void *)(base + off), (lds_void *)dst, 16, 0, 0);
    } else {
        const int q = l - Sh::kA - Sh::kB;
        uint32_t *dst = reinterpret_cast<uint32_t *>(st + Sh::kCodes) + 64 * (wave + kWaves * q);
        const uint8_t *base = q < BM / 32 / kWaves ? g.sa + j * g.sa_step : g.sb + j * g.sb_step;
        __builtin_amdgcn_global_load_lds((global_void *)(base + g.soff[q]), (lds_void *)dst, 4, 0, 0);
    }
}

// What a lane holds of a stage: fragments by K step parity, and scales.
template <int TM, int TN>
struct Frags {
    v4i x[2][TM], w[2][TN];
    uint32_t sx[TM], sw[TN];
};

// One K stage: multiply the stage held in `rd` while (AHEAD) loading stage j
// into `wr`, and (unless LAST) read the first fragments of the next stage from
// `nx`. The barrier sits before the last K step: by then every wavefront has
// read all of this stage's fragments, and the next stage's first ones are read
// while the last step multiplies. Per K step, the next step's fragment reads
// go out in two bursts after the first two MFMAs and one load follows each
// further MFMA; the order is pinned, as a burst of loads would hold the MFMAs.
// The code is one straight line (whole stages are peeled instead of branching
// around loads): the compiler moves these MFMAs across branches, down to where
// their sums are used, and then keeps every fragment alive.
template <int BM, int BN, int STAGES, bool KTAIL, bool AHEAD, bool LAST, int TM, int TN>
__device__ __forceinline__ void stage(const Loads<BM, BN> &g, const uint4 *__restrict__ rd,
                                      uint4 *__restrict__ wr, const uint4 *__restrict__ nx, int j_ahead,
                                      int wave, int a_frag, int b_frag, int a_scale, int b_scale,
                                      int half, int fswz, v16f (&acc)[TM][TN], Frags<TM, TN> &f) {
    using Sh = Shape<BM, BN>;
    constexpr int NMF = TM * TN;
    // three buffers: the stage being loaded is not the next one read, so its
    // loads may follow the barrier too and the barrier leaves the last ones in
    // flight; two buffers: every load precedes the barrier
    constexpr bool LATE = STAGES == 3;
    constexpr int LSTEPS = LATE ? kSteps : kSteps - 1;
    constexpr int LPK = (Sh::kLoads + LSTEPS - 1) / LSTEPS;
    constexpr int LPRE = LATE ? ((kSteps - 1) * LPK < Sh::kLoads ? (kSteps - 1) * LPK : Sh::kLoads) : 0;
    constexpr int NSLOT = NMF > 2 + LPK ? NMF : 2 + LPK;
    const uint4 *next = STAGES == 2 ? wr : nx;
    uint32_t sx[TM], sw[TN];
#pragma unroll
    for (int kk = 0; kk < kSteps; ++kk) {
        const int p = kk & 1;
        if (kk == kSteps - 1 && !LAST) vm_barrier<AHEAD ? LPRE : 0>();
        const uint4 *src = kk + 1 < kSteps ? rd : next;
        const int ch = (4 * half + (kk + 1) % kSteps) ^ fswz;
#pragma unroll
        for (int q = 0; q < NSLOT; ++q) {
            if (q < NMF) {
                const int i = q / TN, j = q % TN;
                acc[i][j] = mfma_32x32x64(kk, f.w[p][j], f.sw[j], f.x[p][i], f.sx[i], acc[i][j]);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (q < 2 && !(LAST && kk == kSteps - 1)) {
#pragma unroll
                for (int r = q; r < TM + TN; r += 2) {
                    if (r < TM) f.x[p ^ 1][r] = __builtin_bit_cast(v4i, src[a_frag + r * 32 * kChunks + ch]);
                    else f.w[p ^ 1][r - TM] = __builtin_bit_cast(v4i, src[b_frag + (r - TM) * 32 * kChunks + ch]);
                }
                if (kk == kSteps - 1) {
                    const uint32_t *sc = reinterpret_cast<const uint32_t *>(next + Sh::kCodes);
#pragma unroll
                    for (int r = q; r < TM + TN; r += 2) {
                        if (r < TM) sx[r] = sc[a_scale + 64 * r];
                        else sw[r - TM] = sc[b_scale + 64 * (r - TM)];
                    }
                }
            }
            const int l = kk * LPK + (q - 2);
            if (AHEAD && kk < LSTEPS && q >= 2 && q < 2 + LPK && l < Sh::kLoads)
                load_one<BM, BN, KTAIL>(g, l, j_ahead, wr, wave);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if constexpr (!LAST) {
#pragma unroll
        for (int i = 0; i < TM; ++i) f.sx[i] = sx[i];
#pragma unroll
        for (int j = 0; j < TN; ++j) f.sw[j] = sw[j];
    }
}

// The wavefront's 32 x WN outputs of sub-tile row i: staged in its own LDS
// (16-byte chunks permuted by the low row bits), then stored in whole pieces.
template <Epilogue EP, int WN, int TN>
__device__ __forceinline__ void store_rows(const v16f (&acc)[TN], uint4 *mine, void *out, int m0,
                                           int m_end, int nw0, int N, int lane) {
    constexpr int SIZE = EP == kOutF32 ? 4 : 2;
    constexpr int CH = WN * SIZE / 16;   // 16-byte chunks per row
    const int row = lane & 31, half = lane >> 5;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float a0 = acc[j][4 * g], a1 = acc[j][4 * g + 1], a2 = acc[j][4 * g + 2], a3 = acc[j][4 * g + 3];
            if constexpr (EP == kOutF32) {
                mine[row * CH + ((j * 8 + 2 * g + half) ^ (row & (CH - 1)))] =
                    __builtin_bit_cast(uint4, v4f{a0, a1, a2, a3});
            } else {
                const uint2 w = EP == kOutBf16
                    ? make_uint2(w8a8::pack_bf16x2(a0, a1), w8a8::pack_bf16x2(a2, a3))
                    : make_uint2(pack_f16x2(a0, a1), pack_f16x2(a2, a3));
                reinterpret_cast<uint2 *>(mine)[2 * (row * CH + ((j * 4 + g) ^ (row & (CH - 1)))) + half] = w;
            }
        }
#pragma unroll
    for (int it = 0; it < 32 * CH / kWave; ++it) {
        const int q = it * kWave + lane, r = q / CH, c = q % CH;
        const uint4 v = mine[r * CH + (c ^ (r & (CH - 1)))];
        const int m = m0 + r, n = nw0 + c * (16 / SIZE);
        if (m < m_end && n < N)
            w8a8::store16_nt(static_cast<char *>(out) + ((int64_t)m * N + n) * SIZE, v);
    }
}

template <int BM, int BN, int STAGES, bool KTAIL, Epilogue EP>
__global__ __launch_bounds__(kThreads, 1) void tiled_kernel(Operands op, Groups grp, int N, int K,
                                                            int KB, int tiles_m, int tiles_n,
                                                            Output o) {
    using Sh = Shape<BM, BN>;
    constexpr int WM = BM / 2, WN = BN / 2, TM = WM / 32, TN = WN / 32;
    static_assert(STAGES == 2 || STAGES == 3, "double or triple buffering");
    __shared__ uint4 lds[STAGES * Sh::kStage];
    static_assert(kWaves * 32 * WN * 4 <= (int)sizeof(lds), "the staged outputs fit");
    w8a8::lds_poison(lds);
    w8a8::lds_poison_done();

    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / 2, wn = wave % 2;

    // tiles XCD by XCD, in groups of 4 tile rows, so that concurrent tiles
    // share activation and weight rows in one L2
    if (grp.offsets) tiles_m = count_tiles<BM>(grp);
    const int tiles = tiles_m * tiles_n;
    if ((int)blockIdx.x >= tiles) return;
    constexpr int kGroupM = 4;
    const int t = w8a8::xcd_contiguous(blockIdx.x, tiles);
    const int per_group = kGroupM * tiles_n;
    const int first_m = (t / per_group) * kGroupM;
    const int gsize = min(tiles_m - first_m, kGroupM);
    const Tile tile = find_tile<BM>(grp, first_m + (t % per_group) % gsize);
    const int n0 = ((t % per_group) / gsize) * BN;
    if (tile.e < 0) return;

    v16f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = v16f{};

    const int frag_row = lane & 31, half = lane >> 5;
    if (tile.e < grp.E) {
        Loads<BM, BN> g;
        {
            const int lrow = 8 * wave + lane / kChunks;
            g.kc = (lane % kChunks) ^ swz(lrow);
            g.half_k = K / 2;
            g.nk = KB;
            const int rows = tile.m1 - tile.m0;
            // without row_token the tile's own rows, else rows anywhere in xq
            const int64_t row0 = grp.row_token ? 0 : tile.m0;
            g.a = op.xq + row0 * (K / 2);
            g.b = op.wq + ((int64_t)tile.e * N + n0) * (K / 2);
            g.sa = op.xs + row0 * 8;
            g.sb = op.ws + ((int64_t)tile.e * KB * N + n0) * 8;
            g.sa_step = (int64_t)grp.T * 8;
            g.sb_step = (int64_t)N * 8;
            auto a_row = [&](int r) -> uint32_t {
                r = min(r, rows - 1);
                return grp.row_token ? (uint32_t)source_row(grp, tile.m0 + r) : (uint32_t)r;
            };
#pragma unroll
            for (int l = 0; l < Sh::kA; ++l) g.aoff[l] = a_row(lrow + 32 * l) * (uint32_t)(K / 2) + g.kc * 16;
#pragma unroll
            for (int l = 0; l < Sh::kB; ++l)
                g.boff[l] = (uint32_t)min(lrow + 32 * l, N - n0 - 1) * (uint32_t)(K / 2) + g.kc * 16;
#pragma unroll
            for (int q = 0; q < Sh::kScale; ++q) {
                const int f = wave + kWaves * q;  // 32-row fragment, activations first
                const uint32_t r = q < BM / 32 / kWaves ? a_row(32 * f + frag_row)
                                                       : (uint32_t)min(32 * (f - BM / 32) + frag_row, N - n0 - 1);
                g.soff[q] = r * 8 + 4 * half;
            }
        }
        const int a_frag = (wm * WM + frag_row) * kChunks;
        const int b_frag = BM * kChunks + (wn * WN + frag_row) * kChunks;
        const int a_scale = wm * (WM / 32) * 64 + lane, b_scale = (BM / 32 + wn * (WN / 32)) * 64 + lane;
        const int fswz = swz(frag_row);
        Frags<TM, TN> f;

        uint4 *rd = lds, *nx = lds + Sh::kStage, *wr = lds + (STAGES - 1) * Sh::kStage;
#pragma unroll
        for (int l = 0; l < Sh::kLoads; ++l) load_one<BM, BN, KTAIL>(g, l, 0, rd, wave);
        if (STAGES == 3 && g.nk > 1) {
#pragma unroll
            for (int l = 0; l < Sh::kLoads; ++l) load_one<BM, BN, KTAIL>(g, l, 1, nx, wave);
            vm_barrier<Sh::kLoads>();
        } else {
            vm_barrier<0>();
        }
        {
            const int ch = (4 * half) ^ fswz;
            const uint32_t *sc = reinterpret_cast<const uint32_t *>(rd + Sh::kCodes);
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                f.x[0][i] = __builtin_bit_cast(v4i, rd[a_frag + i * 32 * kChunks + ch]);
                f.sx[i] = sc[a_scale + 64 * i];
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                f.w[0][j] = __builtin_bit_cast(v4i, rd[b_frag + j * 32 * kChunks + ch]);
                f.sw[j] = sc[b_scale + 64 * j];
            }
        }
#define MXFP4_STAGE(AHEAD, LAST, J)                                                               \
    stage<BM, BN, STAGES, KTAIL, AHEAD, LAST>(g, rd, wr, nx, J, wave, a_frag, b_frag, a_scale,    \
                                              b_scale, half, fswz, acc, f)
        for (int j = STAGES - 1; j < g.nk; ++j) {
            MXFP4_STAGE(true, false, j);
            uint4 *const done = rd;
            rd = nx;
            nx = STAGES == 3 ? wr : done;
            wr = done;
        }
        if (STAGES == 3 && g.nk > 1) {
            MXFP4_STAGE(false, false, 0);
            rd = nx;
        }
        MXFP4_STAGE(false, true, 0);
#undef MXFP4_STAGE
        __syncthreads();  // all fragment reads done before the epilogue reuses LDS
    }

    const int mw0 = tile.m0 + wm * WM, nw0 = n0 + wn * WN;
    if constexpr (EP == kSwiglu) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; j += 2) {
                const int m = mw0 + i * 32 + frag_row;
                store_swiglu(acc[i][j], acc[i][j + 1], o, m, m < tile.m1, nw0 + 32 * j, half, N, grp.S);
            }
    } else {
        constexpr int SIZE = EP == kOutF32 ? 4 : 2;
        uint4 *mine = lds + wave * (32 * WN * SIZE / 16);
#pragma unroll
        for (int i = 0; i < TM; ++i)
            store_rows<EP, WN, TN>(acc[i], mine, o.out, mw0 + i * 32, tile.m1, nw0, N, lane);
    }
}

template <int BM, int BN, int STAGES, Epilogue EP>
hipError_t launch_epilogue(const Operands &op, const Groups &g, int N, int K, const Output &o,
                           hipStream_t stream) {
    const int KB = (K + kStep - 1) / kStep;
    const int tiles_n = (N + BN - 1) / BN;
    const int64_t tiles_m = most_tiles(g.S, g.E, BM, g.offsets != nullptr);
    const dim3 grid((unsigned)(tiles_m * tiles_n)), block(kThreads);
    if (K % kStep == 0)
        tiled_kernel<BM, BN, STAGES, false, EP><<<grid, block, 0, stream>>>(op, g, N, K, KB, (int)tiles_m, tiles_n, o);
    else
        tiled_kernel<BM, BN, STAGES, true, EP><<<grid, block, 0, stream>>>(op, g, N, K, KB, (int)tiles_m, tiles_n, o);
    return hipGetLastError();
}

template <int BM, int BN, int STAGES>
hipError_t launch_shape(const Operands &op, const Groups &g, int N, int K, int epilogue,
                        const Output &o, hipStream_t stream) {
    switch (epilogue) {
        case kOutBf16: return launch_epilogue<BM, BN, STAGES, kOutBf16>(op, g, N, K, o, stream);
        case kOutF16: return launch_epilogue<BM, BN, STAGES, kOutF16>(op, g, N, K, o, stream);
        case kOutF32: return launch_epilogue<BM, BN, STAGES, kOutF32>(op, g, N, K, o, stream);
        default: return launch_epilogue<BM, BN, STAGES, kSwiglu>(op, g, N, K, o, stream);
    }
}

}  // namespace

hipError_t launch_gemm_tiled(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq,
                             const uint8_t *ws, const Groups &g, int N, int K, int epilogue,
                             const Output &o, hipStream_t stream) {
    const Operands op{xq, xs, wq, ws};
    const int64_t t256 = most_tiles(g.S, g.E, 256, g.offsets != nullptr) * ((N + 255) / 256);
    const int64_t t128 = most_tiles(g.S, g.E, 256, g.offsets != nullptr) * ((N + 127) / 128);
    if (t256 >= 4 * 256) return launch_shape<256, 256, 2>(op, g, N, K, epilogue, o, stream);
    if (t128 >= 256) return launch_shape<256, 128, 3>(op, g, N, K, epilogue, o, stream);
    return launch_shape<128, 128, 3>(op, g, N, K, epilogue, o, stream);
}

}  // namespace mxfp4
