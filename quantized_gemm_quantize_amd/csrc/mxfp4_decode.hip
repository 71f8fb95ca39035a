// Weight-streaming MXFP4 products: a dense layer of up to 32 rows, or of more in parts
// of 64 while that fills the CUs better than tiles, or groups of a few rows each
// (product_form in mxfp4_gemm.hip).
//
// With few rows the kernel is bound by reading each weight in use from HBM, once for
// every 16 MT rows. A workgroup owns 16 CT channels of one group's weight and up to 16 MT
// of its rows; its WAVES wavefronts split K in pairs of 128 bytes of codes (256
// elements), wavefront w taking pairs w, w + WAVES, ..., so that neighbouring
// wavefronts read neighbouring cache lines. Measured: 1 x 4096 x 4096 (8.9
// MB) 4.0 us back to back, 5.5 alone; 32 experts' gate and up [4096, 4096] for 64 tokens
// (285 MB) 44-48 us, 6.5-5.9 TB/s; their down products (142 MB) 24.5-26.5 us; one token's
// four experts 9.2 and 4.5 us (36 and 18 MB), where the start and the end of one
// workgroup per CU show.
//
//  - Codes of weights and activations travel global -> LDS with 16-byte
//    direct-to-LDS loads of 8 whole lines each, two pairs in flight per
//    wavefront, into LDS that only this wavefront touches: the mainloop has no
//    barrier. Slot i of a load holds row 8h + i / 8, chunk
//    (i % 8) ^ (i / 8) ^ h, so that fragment reads meet distinct banks.
//  - v_mfma_scale_f32_16x16x128_f8f6f4, twice per pair: lane l holds row l % 16
//    and, in product t, block 2 (l / 16) + t of the pair's eight; its two scale
//    bytes are one 16-bit load.
//  - Blocks past K are read from inside the row; their scale codes are the
//    storage's padding 0 on both sides, and add nothing.
//  - The wavefronts' partial sums are joined in LDS in a fixed order. SwiGLU
//    needs whole blocks of 32 hidden units: CT = 4, 64 channels.
#include "launch.hpp"
#include "mxfp4_epilogue.hpp"
#include "mxfp4_form.hpp"

namespace mxfp4 {
namespace {

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) void global_void;

__device__ __forceinline__ v4f mfma_16x16x128(int sel, v4i a, uint32_t sa, v4i b, uint32_t sb, v4f c) {
    if (sel == 0)
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(a), widen(b), c, kFp4, kFp4, 0, (int)sa, 0, (int)sb);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(a), widen(b), c, kFp4, kFp4, 1, (int)sa, 1, (int)sb);
}

// Activations that are quantized on the way (the single-launch layer): 64
// consecutive elements of a row per lane and pair, its two blocks.
constexpr int kCodes = -1;  // activations in MXFP4 already

template <int XD>
struct RawPair {
    static constexpr int kLoads = XD == kCodes ? 0 : XD == kF32 ? 16 : 8;
    uint4 u[kLoads > 0 ? kLoads : 1];

    // block t of the two -> its scale code, its elements
    __device__ __forceinline__ uint32_t quantize(int t, v4i &x) const {
        uint32_t c[4] = {0, 0, 0, 0};
        uint32_t code = 0;
        if constexpr (XD == kF32) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 &v = u[8 * t + i];
                top = max(top, max(max(v.x & 0x7FFFFFFFu, v.y & 0x7FFFFFFFu), max(v.z & 0x7FFFFFFFu, v.w & 0x7FFFFFFFu)));
            }
            code = scale_code(__uint_as_float(top));
            const float s = scale_value(code);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float *f = reinterpret_cast<const float *>(&u[8 * t + 2 * i]);
                c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[i], f[0], f[1], s, 0);
                c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[i], f[2], f[3], s, 1);
                const float *h = reinterpret_cast<const float *>(&u[8 * t + 2 * i + 1]);
                c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[i], h[0], h[1], s, 2);
                c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c[i], h[2], h[3], s, 3);
            }
        } else if constexpr (XD != kCodes) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 &v = u[4 * t + i];
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    top = max(top, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
            }
            code = scale_code(XD == kBf16 ? __uint_as_float(top << 16)
                                          : (float)__builtin_bit_cast(_Float16, (unsigned short)top));
            const float s = scale_value(code);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 &v = u[4 * t + i];
                if constexpr (XD == kBf16) {
                    using w8a8::v2bf;
                    c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c[i], __builtin_bit_cast(v2bf, v.x), s, 0);
                    c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c[i], __builtin_bit_cast(v2bf, v.y), s, 1);
                    c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c[i], __builtin_bit_cast(v2bf, v.z), s, 2);
                    c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c[i], __builtin_bit_cast(v2bf, v.w), s, 3);
                } else {
                    c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c[i], __builtin_bit_cast(v2h, v.x), s, 0);
                    c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c[i], __builtin_bit_cast(v2h, v.y), s, 1);
                    c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c[i], __builtin_bit_cast(v2h, v.z), s, 2);
                    c[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c[i], __builtin_bit_cast(v2h, v.w), s, 3);
                }
            }
        }
        x = code == 255 ? v4i{} : v4i{(int)c[0], (int)c[1], (int)c[2], (int)c[3]};
        return code;
    }
};

// Waits for a register's load, and with it for the direct-to-LDS loads issued
// before (loads return in order). The compiler's own wait for those is not
// enough where some of the loads in flight are behind a branch.
__device__ __forceinline__ void landed(uint32_t &v) { asm volatile("" : "+v"(v)::"memory"); }

// Waits for this wavefront's LDS reads: a buffer may then be filled again.
__device__ __forceinline__ void fragments_read() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));  // lgkmcnt 0
    asm volatile("" ::: "memory");
}

// One pair in flight: its scales (and activations that have no codes yet).
template <int MT, int CT, int XD>
struct Pair {
    uint32_t sw[CT], sx[MT];
    RawPair<XD> raw;
};

template <int MT, int CT, int WAVES, int XD, Epilogue EP>
__global__ __launch_bounds__(WAVES *kWave) void decode_kernel(
    const uint8_t *__restrict__ xq, const uint8_t *__restrict__ xs, const uint8_t *__restrict__ wq,
    const uint8_t *__restrict__ ws, Groups grp, int N, int K, int KB, int tiles_n, int64_t ldx, Ids slots, Output o) {
    static_assert(XD == kCodes || MT == 1, "up to 16 rows are quantized on the way");
    constexpr int XT = XD == kCodes ? MT : 0;        // 16-row tiles of codes in LDS
    constexpr int kSlots = WAVES * (XT + CT) * 128;  // 16-byte slots of one pair, all wavefronts
    // one array per pair in flight: the compiler then waits for that pair only
    __shared__ uint4 q0[kSlots], q1[kSlots];
    static_assert(WAVES * MT * CT * kWave <= kSlots, "the partial sums fit a pair's place");
    w8a8::lds_poison(q0);
    w8a8::lds_poison(q1);
    w8a8::lds_poison_done();

    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    Tile t;
    int64_t xbase = 0;  // first row of the activations that are quantized on the way
    if (XD != kCodes && slots.ids) {
        // unsorted slots, one row each
        const int slot = blockIdx.x / tiles_n;
        t = Tile{expert_of(slots, slot, grp.E), slot, slot + 1};
        xbase = slot / slots.top;
    } else {
        const int tile = blockIdx.x / tiles_n;
        const Group own = find_group<16 * MT>(grp, grp.offsets ? scan_groups<16 * MT>(grp, 0) : GroupScan{}, tile);
        t = Tile{own.e, own.lo + (tile - own.first) * 16 * MT, own.lo + own.n};
    }
    if (t.e < 0) return;
    const int n0 = (blockIdx.x % tiles_n) * 16 * CT;
    const int rows = t.m1 - t.m0;
    const bool weight = t.e < grp.E;

    v4f acc[MT][CT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[m][c] = v4f{};
    const int r16 = lane & 15, quarter = lane >> 4;
    if (weight) {
        const int lr = lane >> 3, lc = lane & 7;
        int row[3 * MT];  // per 16-row tile: the rows of this lane's two code loads, of its scales
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            row[3 * m] = t.m0 + min(16 * m + lr, rows - 1);
            row[3 * m + 1] = t.m0 + min(16 * m + 8 + lr, rows - 1);
            row[3 * m + 2] = t.m0 + min(16 * m + r16, rows - 1);
        }
        if (XD == kCodes && grp.row_token) source_rows(grp, row);
        const uint8_t *wrow[CT][2], *xrow[MT][2], *wsc[CT], *xsc[MT];
        int chunk[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            chunk[h] = lc ^ lr ^ h;
#pragma unroll
            for (int c = 0; c < CT; ++c)
                wrow[c][h] = wq + ((int64_t)t.e * N + min(n0 + 16 * c + 8 * h + lr, N - 1)) * (K / 2);
#pragma unroll
            for (int m = 0; m < XT; ++m) xrow[m][h] = xq + (int64_t)row[3 * m + h] * (K / 2);
        }
#pragma unroll
        for (int c = 0; c < CT; ++c)
            wsc[c] = ws + ((int64_t)t.e * KB * N + min(n0 + 16 * c + r16, N - 1)) * 8 + 2 * quarter;
#pragma unroll
        for (int m = 0; m < XT; ++m) xsc[m] = xs + (int64_t)row[3 * m + 2] * 8 + 2 * quarter;

        auto load = [&](int p, uint4 *q, Pair<MT, CT, XD> &s) {
            uint4 *mine = q + wave * (XT + CT) * 128;
            int at[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)  // a chunk past K: the pair's first one
                at[h] = p * kStepBytes + (p * kStepBytes + chunk[h] * 16 < K / 2 ? chunk[h] * 16 : 0);
            if constexpr (XD != kCodes) {
                // before the weights: it lands first, and is quantized while they travel
                constexpr int kPer = XD == kF32 ? 4 : 8;  // elements per load
                const int k = p * kStep + 64 * quarter;
                const char *x = reinterpret_cast<const char *>(xq) + ((xbase + r16) * ldx + k) * (16 / kPer);
#pragma unroll
                for (int i = 0; i < RawPair<XD>::kLoads; ++i)
                    s.raw.u[i] = r16 < rows && k + kPer * i < K ? *reinterpret_cast<const uint4 *>(x + 16 * i)
                                                                : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    __builtin_amdgcn_global_load_lds((global_void *)(wrow[c][h] + at[h]),
                                                     (lds_void *)(mine + 128 * (XT + c) + 64 * h), 16, 0,
                                                     w8a8::kLdsLoadStream);
#pragma unroll
            for (int m = 0; m < XT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    __builtin_amdgcn_global_load_lds((global_void *)(xrow[m][h] + at[h]),
                                                     (lds_void *)(mine + 128 * m + 64 * h), 16, 0, 0);
            asm volatile("" ::: "memory");  // the scales' loads stay behind these
#pragma unroll
            for (int m = 0; m < XT; ++m) s.sx[m] = *reinterpret_cast<const uint16_t *>(xsc[m] + (int64_t)p * grp.T * 8);
#pragma unroll
            for (int c = 0; c < CT; ++c) s.sw[c] = *reinterpret_cast<const uint16_t *>(wsc[c] + (int64_t)p * N * 8);
        };
        auto multiply = [&](const uint4 *q, Pair<MT, CT, XD> &s) {
            const uint4 *mine = q + wave * (XT + CT) * 128;
#pragma unroll
            for (int c = 0; c < CT; ++c) landed(s.sw[c]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int slot = (r16 >> 3) * 64 + (r16 & 7) * 8 + ((2 * quarter + u) ^ (r16 & 7) ^ (r16 >> 3));
                v4i w[CT];
#pragma unroll
                for (int c = 0; c < CT; ++c) w[c] = __builtin_bit_cast(v4i, mine[128 * (XT + c) + slot]);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    v4i x;
                    uint32_t sx;
                    if constexpr (XD == kCodes) {
                        x = __builtin_bit_cast(v4i, mine[128 * m + slot]);
                        sx = s.sx[m];
                    } else {
                        sx = s.raw.quantize(u, x) << (8 * u);
                    }
#pragma unroll
                    for (int c = 0; c < CT; ++c) acc[m][c] = mfma_16x16x128(u, w[c], s.sw[c], x, sx, acc[m][c]);
                }
            }
        };
        Pair<MT, CT, XD> s0, s1;
        int p = wave;
        if (p < KB) load(p, q0, s0);
        if (p + WAVES < KB) load(p + WAVES, q1, s1);
        for (; p < KB; p += 2 * WAVES) {
            multiply(q0, s0);
            fragments_read();
            if (p + 2 * WAVES < KB) load(p + 2 * WAVES, q0, s0);
            if (p + WAVES < KB) multiply(q1, s1);
            fragments_read();
            if (p + 3 * WAVES < KB) load(p + 3 * WAVES, q1, s1);
        }
    }

    // acc[m][c], element i of lane l: row 16 m + l % 16, channel 16 c + 4 (l / 16) + i
    __syncthreads();  // every wavefront has read its last fragments
    v4f(*red)[MT * CT][kWave] = reinterpret_cast<v4f(*)[MT * CT][kWave]>(q0);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < CT; ++c) red[wave][m * CT + c][lane] = acc[m][c];
    __syncthreads();
    if constexpr (EP != kSwiglu) {
        // one thread: 4 channels of a row
        for (int e = threadIdx.x; e < MT * CT * kWave; e += WAVES * kWave) {
            const int tile = e / kWave, l = e % kWave;
            v4f sum = red[0][tile][l];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) {
                const v4f v = red[w][tile][l];
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] += v[i];
            }
            const int m = 16 * (tile / CT) + (l & 15), n = n0 + 16 * (tile % CT) + 4 * (l >> 4);
            if (m >= rows || n >= N) continue;
            const int64_t at = (int64_t)(t.m0 + m) * N + n;
            if constexpr (EP == kOutF32)
                *reinterpret_cast<v4f *>(static_cast<float *>(o.out) + at) = sum;
            else if constexpr (EP == kOutBf16)
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(o.out) + at) =
                    make_uint2(w8a8::pack_bf16x2(sum[0], sum[1]), w8a8::pack_bf16x2(sum[2], sum[3]));
            else
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(o.out) + at) =
                    make_uint2(pack_f16x2(sum[0], sum[1]), pack_f16x2(sum[2], sum[3]));
        }
    } else {
        static_assert(CT == 4 || EP != kSwiglu, "a block of 32 hidden units");
        // one thread: 4 channels, i.e. hidden units 2 u and 2 u + 1 of the block
        // with u = 4 c + l / 16; 16 threads share a row's block
        const int F = N / 2, f0 = n0 / 2;
        for (int e = threadIdx.x; e < MT * 16 * 16; e += WAVES * kWave) {
            const int m = e >> 4, u = e & 15;  // row of the tile, pair of hidden units
            const int l = (m & 15) + 16 * (u & 3), tile = (m >> 4) * CT + (u >> 2);
            v4f sum = red[0][tile][l];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) {
                const v4f v = red[w][tile][l];
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] += v[i];
            }
            const float h0 = swiglu(sum[0], sum[1]), h1 = swiglu(sum[2], sum[3]);
            uint32_t top = max(__float_as_uint(h0) & 0x7FFFFFFFu, __float_as_uint(h1) & 0x7FFFFFFFu);
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, kWave));
            const uint32_t code = scale_code(__uint_as_float(top));
            uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, h0, h1, scale_value(code), 0) & 0xFFu;
            if (code == 255) c = 0;
            if (m >= rows || f0 >= F) continue;
            const int64_t row = t.m0 + m;
            o.codes[row * (F / 2) + f0 / 2 + u] = (uint8_t)c;
            if (u == 0) {
                uint8_t *s = o.scales + ((int64_t)(f0 / kStep) * grp.S + row) * 8;
                const int b = (f0 / 32) % 8;
                s[b] = (uint8_t)code;
                if (f0 + 32 == F)
                    for (int i = b + 1; i < 8; ++i) s[i] = 0;
            }
        }
    }
}

// The down products of a few tokens and their weighted sum, without a sort: a
// workgroup owns 16 channels of one token and runs through its slots' weights
// (hidden rows in slot order), its wavefronts splitting slots and K. Each pair's
// products are weighted and added in fp32; slots without an expert are left out.
constexpr int kDownWaves = 8;

template <Dtype D>
__global__ __launch_bounds__(kDownWaves *kWave) void down_combine_kernel(
    const uint8_t *__restrict__ hq, const uint8_t *__restrict__ hs, const uint8_t *__restrict__ wq,
    const uint8_t *__restrict__ ws, Ids slots, const float *__restrict__ weights, int S, int E, int N,
    int K, int KB, int tiles_n, void *__restrict__ out) {
    __shared__ uint4 q0[kDownWaves * 128], q1[kDownWaves * 128], q2[kDownWaves * 128], q3[kDownWaves * 128];
    w8a8::lds_poison(q0);
    w8a8::lds_poison(q1);
    w8a8::lds_poison(q2);
    w8a8::lds_poison(q3);
    w8a8::lds_poison_done();
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t token = blockIdx.x / tiles_n;
    const int n0 = (blockIdx.x % tiles_n) * 16;  // N is a multiple of 16
    const int r16 = lane & 15, quarter = lane >> 4, lr = lane >> 3, lc = lane & 7;

    // lane j: slot j's expert and weight (a load of its own in each item's chain
    // would wait for all loads before it)
    const int64_t own = token * slots.top + min(lane, slots.top - 1);
    uint32_t slot_weight = __float_as_uint(weights[own]);
    const int slot_expert = expert_of(slots, own, E);
    landed(slot_weight);
    struct Item {
        uint32_t sw, sx;
        uint4 x[2];
        float weight;
        bool live;
    };
    auto load = [&](int item, uint4 *q, Item &s) {
        const int j = item / KB, p = item % KB;
        const int64_t slot = token * slots.top + j;
        const int e = __builtin_amdgcn_readlane(slot_expert, j);
        s.live = e < E;
        if (!s.live) return;
        s.weight = __uint_as_float(__builtin_amdgcn_readlane(slot_weight, j));
        const int k16 = p * 8 + 2 * quarter;  // 16-byte chunks along K; one past K: the row's first
        const uint4 *x = reinterpret_cast<const uint4 *>(hq + slot * (K / 2));
#pragma unroll
        for (int u = 0; u < 2; ++u) s.x[u] = x[(k16 + u) * 16 < K / 2 ? k16 + u : 0];
        s.sx = *reinterpret_cast<const uint16_t *>(hs + ((int64_t)p * S + slot) * 8 + 2 * quarter);
        uint4 *mine = q + wave * 128;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int chunk = (lc ^ lr ^ h) * 16;  // one past K: the pair's first
            const int at = p * kStepBytes + (p * kStepBytes + chunk < K / 2 ? chunk : 0);
            __builtin_amdgcn_global_load_lds((global_void *)(wq + ((int64_t)e * N + n0 + 8 * h + lr) * (K / 2) + at),
                                             (lds_void *)(mine + 64 * h), 16, 0, w8a8::kLdsLoadStream);
        }
        asm volatile("" ::: "memory");  // the scale's load stays behind these
        s.sw = *reinterpret_cast<const uint16_t *>(ws + (((int64_t)e * KB + p) * N + n0 + r16) * 8 + 2 * quarter);
    };
    v4f sum = {};
    auto multiply = [&](const uint4 *q, Item &s) {
        if (!s.live) return;
        const uint4 *mine = q + wave * 128;
        landed(s.sw);
        v4f acc = {};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int slot = (r16 >> 3) * 64 + (r16 & 7) * 8 + ((2 * quarter + u) ^ (r16 & 7) ^ (r16 >> 3));
            // one row of activations: the lanes of the other fifteen hold zeros
            const v4i x = r16 == 0 ? __builtin_bit_cast(v4i, s.x[u]) : v4i{};
            acc = mfma_16x16x128(u, __builtin_bit_cast(v4i, mine[slot]), s.sw, x, s.sx, acc);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += s.weight * acc[i];
    };
    const int items = slots.top * KB;
    Item s0{}, s1{}, s2{}, s3{};
    int i = wave;
    if (i < items) load(i, q0, s0);
    if (i + kDownWaves < items) load(i + kDownWaves, q1, s1);
    if (i + 2 * kDownWaves < items) load(i + 2 * kDownWaves, q2, s2);
    if (i + 3 * kDownWaves < items) load(i + 3 * kDownWaves, q3, s3);
    for (; i < items; i += 4 * kDownWaves) {
        multiply(q0, s0);
        fragments_read();
        if (i + 4 * kDownWaves < items) load(i + 4 * kDownWaves, q0, s0);
        if (i + kDownWaves < items) multiply(q1, s1);
        fragments_read();
        if (i + 5 * kDownWaves < items) load(i + 5 * kDownWaves, q1, s1);
        if (i + 2 * kDownWaves < items) multiply(q2, s2);
        fragments_read();
        if (i + 6 * kDownWaves < items) load(i + 6 * kDownWaves, q2, s2);
        if (i + 3 * kDownWaves < items) multiply(q3, s3);
        fragments_read();
        if (i + 7 * kDownWaves < items) load(i + 7 * kDownWaves, q3, s3);
    }
    __syncthreads();  // every wavefront has read its last fragments
    v4f(*red)[4] = reinterpret_cast<v4f(*)[4]>(q0);
    if (r16 == 0) red[wave][quarter] = sum;  // row 0: channels 4 quarter .. + 3
    __syncthreads();
    if (threadIdx.x < 16) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kDownWaves; ++w) v += red[w][threadIdx.x >> 2][threadIdx.x & 3];
        const int64_t at = token * N + n0 + threadIdx.x;
        if constexpr (D == kF32) static_cast<float *>(out)[at] = v;
        else if constexpr (D == kBf16) static_cast<__bf16 *>(out)[at] = (__bf16)v;
        else static_cast<_Float16 *>(out)[at] = (_Float16)v;
    }
}

template <int MT, int CT, int WAVES, Epilogue EP>
hipError_t launch_ep(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws,
                     const Groups &g, int N, int K, const Output &o, hipStream_t stream) {
    const int KB = (K + kStep - 1) / kStep, tiles_n = (N + 16 * CT - 1) / (16 * CT);
    const int64_t tiles = most_tiles(g.S, g.E, 16 * MT, g.offsets != nullptr) * tiles_n;
    decode_kernel<MT, CT, WAVES, kCodes, EP><<<dim3((unsigned)tiles), dim3(WAVES * kWave), 0, stream>>>(
        xq, xs, wq, ws, g, N, K, KB, tiles_n, 0, Ids{}, o);
    return hipGetLastError();
}

template <int MT, int CT, int WAVES>
hipError_t launch_plain(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws,
                        const Groups &g, int N, int K, int epilogue, const Output &o, hipStream_t stream) {
    switch (epilogue) {
        case kOutBf16: return launch_ep<MT, CT, WAVES, kOutBf16>(xq, xs, wq, ws, g, N, K, o, stream);
        case kOutF16: return launch_ep<MT, CT, WAVES, kOutF16>(xq, xs, wq, ws, g, N, K, o, stream);
        default: return launch_ep<MT, CT, WAVES, kOutF32>(xq, xs, wq, ws, g, N, K, o, stream);
    }
}

template <int MT>
hipError_t launch_rows(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws,
                       const Groups &g, int N, int K, int epilogue, const Output &o, const Form &f,
                       hipStream_t stream) {
    if constexpr (MT < 4) {
        if (epilogue == kSwiglu)
            return f.waves == 4 ? launch_ep<MT, 4, 4, kSwiglu>(xq, xs, wq, ws, g, N, K, o, stream)
                                : launch_ep<MT, 4, 2, kSwiglu>(xq, xs, wq, ws, g, N, K, o, stream);
        if (f.channels == 64) return launch_plain<MT, 4, 2>(xq, xs, wq, ws, g, N, K, epilogue, o, stream);
        if (f.channels == 32) return launch_plain<MT, 2, 4>(xq, xs, wq, ws, g, N, K, epilogue, o, stream);
        return launch_plain<MT, 1, 8>(xq, xs, wq, ws, g, N, K, epilogue, o, stream);
    } else {
        return launch_plain<MT, 1, 4>(xq, xs, wq, ws, g, N, K, epilogue, o, stream);
    }
}

template <int XD, Epilogue EP>
hipError_t launch_fused(const void *x, int64_t ldx, const uint8_t *wq, const uint8_t *ws, int M, int N,
                        int K, const Output &o, hipStream_t stream) {
    const int tiles_n = (N + 15) / 16;
    decode_kernel<1, 1, 8, XD, EP><<<dim3((unsigned)tiles_n), dim3(8 * kWave), 0, stream>>>(
        static_cast<const uint8_t *>(x), nullptr, wq, ws, Groups{nullptr, nullptr, 1, M, M}, N, K,
        (K + kStep - 1) / kStep, tiles_n, ldx, Ids{}, o);
    return hipGetLastError();
}

template <int XD>
hipError_t launch_fused(const void *x, int64_t ldx, const uint8_t *wq, const uint8_t *ws, int M, int N,
                        int K, int out_dtype, const Output &o, hipStream_t stream) {
    switch (out_dtype) {
        case kBf16: return launch_fused<XD, kOutBf16>(x, ldx, wq, ws, M, N, K, o, stream);
        case kF16: return launch_fused<XD, kOutF16>(x, ldx, wq, ws, M, N, K, o, stream);
        default: return launch_fused<XD, kOutF32>(x, ldx, wq, ws, M, N, K, o, stream);
    }
}

template <int WAVES, int XD>
hipError_t launch_slots(const void *x, int64_t ldx, const Ids &slots, int S, int E, const uint8_t *wq,
                        const uint8_t *ws, int F, int K, uint8_t *hq, uint8_t *hs, hipStream_t stream) {
    const int N = 2 * F, tiles_n = (N + 63) / 64;
    decode_kernel<1, 4, WAVES, XD, kSwiglu><<<dim3((unsigned)(S * tiles_n)), dim3(WAVES * kWave), 0, stream>>>(
        static_cast<const uint8_t *>(x), nullptr, wq, ws, Groups{nullptr, nullptr, E, S, S}, N, K,
        (K + kStep - 1) / kStep, tiles_n, ldx, slots, Output{nullptr, hq, hs});
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_decode(const void *x, int64_t ldx, int x_dtype, int M, const uint8_t *wq,
                                const uint8_t *ws, int N, int K, int out_dtype, void *out,
                                hipStream_t stream) {
    const Output o{out, nullptr, nullptr};
    switch (x_dtype) {
        case kBf16: return launch_fused<kBf16>(x, ldx, wq, ws, M, N, K, out_dtype, o, stream);
        case kF16: return launch_fused<kF16>(x, ldx, wq, ws, M, N, K, out_dtype, o, stream);
        default: return launch_fused<kF32>(x, ldx, wq, ws, M, N, K, out_dtype, o, stream);
    }
}

hipError_t launch_moe_up(const void *x, int64_t ldx, int dtype, const Ids &slots, int S, int E,
                         const uint8_t *wq, const uint8_t *ws, int F, int K, uint8_t *hq, uint8_t *hs,
                         hipStream_t stream) {
    // 8 wavefronts have all of a workgroup's weights under way at once: where no
    // CU has a second workgroup to fill the time (1 token, 4 experts of
    // 4096 / 2048: the layer 18.2 -> 17.6 us; 2 tokens 25.7 -> 28.3)
    const int KB = (K + kStep - 1) / kStep;
    const bool wide = KB >= 8 && (int64_t)S * ((2 * F + 63) / 64) <= w8a8::device_cu_count();
    switch (dtype) {
        case kBf16:
            return wide ? launch_slots<8, kBf16>(x, ldx, slots, S, E, wq, ws, F, K, hq, hs, stream)
                        : launch_slots<4, kBf16>(x, ldx, slots, S, E, wq, ws, F, K, hq, hs, stream);
        case kF16:
            return wide ? launch_slots<8, kF16>(x, ldx, slots, S, E, wq, ws, F, K, hq, hs, stream)
                        : launch_slots<4, kF16>(x, ldx, slots, S, E, wq, ws, F, K, hq, hs, stream);
        default: return launch_slots<4, kF32>(x, ldx, slots, S, E, wq, ws, F, K, hq, hs, stream);
    }
}

hipError_t launch_moe_down(const uint8_t *hq, const uint8_t *hs, const Ids &slots, const float *weights,
                           int T, int E, const uint8_t *wq, const uint8_t *ws, int N, int K, int dtype,
                           void *out, hipStream_t stream) {
    const int KB = (K + kStep - 1) / kStep, tiles_n = N / 16, S = T * slots.top;
    const dim3 grid((unsigned)(T * tiles_n)), block(kDownWaves * kWave);
    switch (dtype) {
        case kBf16: down_combine_kernel<kBf16><<<grid, block, 0, stream>>>(hq, hs, wq, ws, slots, weights, S, E, N, K, KB, tiles_n, out); break;
        case kF16: down_combine_kernel<kF16><<<grid, block, 0, stream>>>(hq, hs, wq, ws, slots, weights, S, E, N, K, KB, tiles_n, out); break;
        default: down_combine_kernel<kF32><<<grid, block, 0, stream>>>(hq, hs, wq, ws, slots, weights, S, E, N, K, KB, tiles_n, out);
    }
    return hipGetLastError();
}

hipError_t launch_gemm_decode(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq,
                              const uint8_t *ws, const Groups &g, int N, int K, int epilogue,
                              const Output &o, const Form &f, hipStream_t stream) {
    if (f.rows == 16) return launch_rows<1>(xq, xs, wq, ws, g, N, K, epilogue, o, f, stream);
    if (f.rows == 32) return launch_rows<2>(xq, xs, wq, ws, g, N, K, epilogue, o, f, stream);
    return launch_rows<4>(xq, xs, wq, ws, g, N, K, epilogue, o, f, stream);
}

}  // namespace mxfp4
