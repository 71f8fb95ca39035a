// MXFP4 building blocks shared by the kernels (gfx950 / CDNA4).
//
// A row is cut into blocks of 32 elements along K. Each block holds 4-bit
// e2m1 elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) and one
// power-of-two scale stored as a biased exponent (e8m0: 2^(code - 127), code
// 255 is NaN).
//   codes  [rows, K/2]            byte j of a row: element 2j in the low nibble
//   scales [ceil(K/256), rows, 8] byte i of (b, row): the scale of block 8b+i,
//                                 0 past the row's last block
// The scales are K-block-major so that the 8 scale bytes that a product needs
// per row and 256-element step lie next to those of the neighbouring rows: a
// 32-row fragment's scales are one 256-byte load.
#pragma once

#include "common.hpp"

namespace mxfp4 {

using w8a8::kWave;
using w8a8::v4i;

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

enum Dtype { kBf16 = 0, kF16 = 1, kF32 = 2 };

constexpr int kFp4 = 4;        // operand format selector of the scaled MFMA
constexpr int kStep = 256;     // elements per scale group of 8 blocks
constexpr int kStepBytes = 128;

// The float behind a scale code: 2^(code - 127), 2^-127 for code 0, NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t code) {
    return __uint_as_float(code == 0 ? 0x00400000u : code == 255 ? 0x7FC00000u : code << 23);
}

// Scale code of a block whose largest magnitude is `top`: floor(log2 top) - 2
// (2 is the exponent of the largest element, 6 = 1.5 * 2^2), at least -127;
// 255 when the block holds a value that is not finite.
__device__ __forceinline__ uint32_t scale_code(float top) {
    const uint32_t field = __float_as_uint(top) >> 23;  // top >= 0
    return field == 255 ? 255u : field < 2 ? 0u : field - 2;
}

__device__ __forceinline__ v8i widen(v4i a) {
    // the fp4 forms read the first four registers of the operand
    return __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
}

// Scaled fp4 MFMA, 32x32 output, K = 64: lane l holds row l % 32 of each
// operand, 32 consecutive elements (block l / 32 of the two), and byte SEL of
// its scale register is that block's scale. Output as the int8 form: lane l,
// element r: row 8 * (r / 4) + 4 * (l / 32) + r % 4 of a, row l % 32 of b.
template <int SEL>
__device__ __forceinline__ v16f mfma_32x32x64(v4i a, uint32_t sa, v4i b, uint32_t sb, v16f c) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(a), widen(b), c, kFp4, kFp4, SEL,
                                                           (int)sa, SEL, (int)sb);
}

// The same with the byte chosen by a loop counter (constant once unrolled).
__device__ __forceinline__ v16f mfma_32x32x64(int sel, v4i a, uint32_t sa, v4i b, uint32_t sb,
                                              v16f c) {
    switch (sel) {
        case 0: return mfma_32x32x64<0>(a, sa, b, sb, c);
        case 1: return mfma_32x32x64<1>(a, sa, b, sb, c);
        case 2: return mfma_32x32x64<2>(a, sa, b, sb, c);
        default: return mfma_32x32x64<3>(a, sa, b, sb, c);
    }
}

// Rows of the product, in groups: rows offsets[e] .. offsets[e+1]-1 multiply
// weight e; rows past offsets[E] belong to no weight (their outputs are 0).
// offsets null: one group of all S rows. Row r reads activation row
// row_token[r] of T (row_token null: row r itself).
struct Groups {
    const int32_t *offsets;
    const int32_t *row_token;
    int E, S, T;
};

// Expert ids of slots, `top` per token, 32 or 64 bits each.
struct Ids {
    const void *ids;
    int bits, top;
};

// Expert of a slot, E when its id names none.
__device__ __forceinline__ int expert_of(const Ids &s, int64_t slot, int E) {
    const int64_t id = s.bits == 64 ? static_cast<const int64_t *>(s.ids)[slot]
                                    : static_cast<const int32_t *>(s.ids)[slot];
    return id >= 0 && id < E ? (int)id : E;
}

struct Tile {
    int e;       // group, E for the rows without a weight, -1 past the last tile
    int m0, m1;  // its rows: m0 .. m1-1 with m1 the end of the group
};

// Inclusive sum over the lanes of a wavefront, in six lane moves of the vector
// unit (shuffles go through LDS: several times their latency, and every
// workgroup of the grouped kernels starts with this).
__device__ __forceinline__ int scan_lanes(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // last lane of rows 0, 2 to 1, 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // lane 31 to rows 2, 3
    return v;
}

// 64 consecutive groups from `base` on, one per lane: the group's first row and
// rows (none past group E, which holds the rows without a weight), and the tiles
// of these groups up to and including it. Bounds that a malformed offsets array
// could break are clamped, so rows stay inside [0, S).
struct GroupScan {
    int lo, n, upto;
};

template <int BM>
__device__ __forceinline__ GroupScan scan_groups(const Groups &g, int base) {
    int e = base + (threadIdx.x & (kWave - 1));
    asm volatile("" : "+v"(e));  // or a persistent kernel keeps the addresses in registers
    int a = g.offsets[min(e, g.E)], b = g.offsets[min(e + 1, g.E)];
    asm volatile("" : "+v"(a), "+v"(b));  // both under way together, not the second one in a branch
    GroupScan s;
    s.lo = min(max(a, 0), g.S);
    s.n = e < g.E ? min(max(b, s.lo), g.S) - s.lo : e == g.E ? g.S - s.lo : 0;
    s.upto = scan_lanes((s.n + BM - 1) / BM);
    return s;
}

// All tiles of BM rows, found by every wavefront for itself (first: the scan
// from group 0 on).
template <int BM>
__device__ __forceinline__ int count_tiles(const Groups &g, const GroupScan &first) {
    int total = __builtin_amdgcn_readlane(first.upto, kWave - 1);
    for (int base = kWave; base <= g.E; base += kWave)
        total += __builtin_amdgcn_readlane(scan_groups<BM>(g, base).upto, kWave - 1);
    return total;
}

// The group that holds tile t of the groups' rows cut into tiles of BM rows,
// group after group, 64 groups at a time.
struct Group {
    int e;      // E for the rows without a weight, -1 past the last tile
    int lo, n;  // first row, rows
    int first;  // its first tile
};

template <int BM>
__device__ __forceinline__ Group find_group(const Groups &g, const GroupScan &first, int t) {
    if (!g.offsets) return Group{t * BM < g.S ? 0 : -1, 0, g.S, 0};
    GroupScan s = first;
    int before = 0;
    for (int base = 0; base <= g.E; base += kWave) {
        if (base > 0) s = scan_groups<BM>(g, base);
        const uint64_t hit = __builtin_amdgcn_ballot_w64(before + s.upto > t);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            const int lo = __builtin_amdgcn_readlane(s.lo, l), n = __builtin_amdgcn_readlane(s.n, l);
            return Group{base + l, lo, n, before + __builtin_amdgcn_readlane(s.upto, l) - (n + BM - 1) / BM};
        }
        before += __builtin_amdgcn_readlane(s.upto, kWave - 1);
    }
    return Group{-1, 0, 0, 0};
}

// Most tiles of BM rows that S rows in E groups (and the rows without a
// weight) can have: every group ends in at most one partial tile, and no tile
// is empty.
inline int64_t most_tiles(int64_t S, int64_t E, int BM, bool grouped) {
    const int64_t full = (S + BM - 1) / BM;
    if (!grouped) return full;
    const int64_t split = S / BM + E + 1;
    return split < S ? split : S;
}

// Activation rows of N product rows: r[i] -> row_token[r[i]], all loads under way
// together.
template <int N>
__device__ __forceinline__ void source_rows(const Groups &g, int (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = g.row_token[r[i]];
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = min(max(r[i], 0), g.T - 1);
}

// Gate and up projections of one hidden unit -> its activation, gate / (1 +
// exp(-gate)) * up. With t = 2^-13 exp(-gate / 2) the sum is 2^26 (t^2 + 2^-26): it
// overflows for no gate above -105, where the sigmoid rounds to 0, and v_rcp_f32
// (within 1 ulp; it flushes results below 2^-126) sees 2^-26 to 2^126, so that gates
// under -87 keep their activations (the sigmoid is then below 2^-126, in steps of
// 2^-149). The 13 in the exponent's argument costs 2^-21 of t at most. The correctly
// rounded division made the epilogue of a 256 x 256 tile several times as long.
constexpr float kHalfLog2e = 0.72134752f;
constexpr float kTwoM26 = 1.0f / 67108864.0f;

__device__ __forceinline__ float swiglu(float gate, float up) {
    const float t = __builtin_amdgcn_exp2f(__builtin_fmaf(-kHalfLog2e, gate, -13.0f));
    const float r = __builtin_amdgcn_rcpf(__builtin_fmaf(t, t, kTwoM26));
    return gate * (r * kTwoM26) * up;
}

// Four at once, step by step: one after the other, each waits for its own
// exponential and reciprocal (32 experts' gate and up of 8192 tokens 318 -> 314 us).
__device__ __forceinline__ v4f swiglu4(const v4f &gate, const v4f &up) {
    float t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(-kHalfLog2e, gate[i], -13.0f));
    asm volatile("" : "+v"(t[0]), "+v"(t[1]), "+v"(t[2]), "+v"(t[3]));
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = __builtin_amdgcn_rcpf(__builtin_fmaf(t[i], t[i], kTwoM26));
    asm volatile("" : "+v"(t[0]), "+v"(t[1]), "+v"(t[2]), "+v"(t[3]));
    v4f v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = gate[i] * (t[i] * kTwoM26) * up[i];
    return v;
}

}  // namespace mxfp4
