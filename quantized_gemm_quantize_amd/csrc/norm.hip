// The step between two blocks of a model: a block's output y joins the
// residual stream, and the stream is normalized for the next block.
//
//   u = y                          or y / rms(y) * post_weight
//   r' = r + scale * gate * u      (gate: none, one value per channel, or a row per token)
//   o = r' / rms(r') * weight      rms(v) = sqrt(sum_h v^2 / H + eps)
//
// r' is written in the rows' type; o is made of the unrounded r' and written in
// that type, or quantized as w8a8_quantize_rows (int8, one scale per row) or
// mxfp4_quantize_rows would quantize the unrounded o: the rows that the
// next product reads, without a pass of their own.
//
// Bound by HBM: y, r (and the gate) are read once and r', o written once, with
// a row in registers between. A row belongs to TPR threads (16 of a wavefront, a
// wavefront, or a workgroup), chunk c * TPR + t of 16 bytes to thread t; both
// sums of squares and the row's largest magnitude are reduced across lanes, and
// through LDS beyond a wavefront. Weights (and a gate vector) are loaded beside the row,
// not after its sums, where registers allow it. Measured: 16448 x 1280 bf16 with post norm and gate
// 39 us (4.3 TB/s), to int8 rows 43 (3.4), 8192 x 4096 without 48 us (5.6 TB/s, part of it held on
// chip by repeated calls), to int8 47 (5.0) and MXFP4 rows 44 (4.9), 32-bit 81 us (6.6); a single row 4 us.
#include "launch.hpp"
#include "norm.hpp"
#include "quant_math.hpp"
#include "rows.hpp"

namespace block {
namespace {

using namespace rows;

// MXFP4 block of 32 elements held by 32 / V neighbouring threads, V each: the
// scale code and this thread's element codes (V / 2 bytes).
template <int V>
__device__ __forceinline__ uint32_t mx_block(const float (&v)[V], uint32_t &codes) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < V; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
#pragma unroll
    for (int off = 1; off < 32 / V; off <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, kWave));
    const uint32_t code = mxfp4::scale_code(__uint_as_float(m));
    const float s = mxfp4::scale_value(code);
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], s, 1);
    if constexpr (V == 8) {
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], s, 2);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], s, 3);
    }
    codes = code == 255 ? 0u : r;
    return code;
}

template <Dtype D, Out O, int TPR, int C, bool WHOLE>
__global__ __launch_bounds__(TPR <= kWave ? 256 : TPR) void norm_kernel(const Forward a) {
    typedef typename Element<D>::type E;
    constexpr int V = kPer<D>;
    constexpr int kThreads = TPR <= kWave ? 256 : TPR;
    constexpr int kRows = kThreads / TPR;
    __shared__ float red[2][kThreads / kWave][1];
    __shared__ uint32_t red_max[kThreads / kWave];
    w8a8::lds_poison(red);
    w8a8::lds_poison(red_max);
    w8a8::lds_poison_done();
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    if (row >= a.T) return;  // uniform per row, and a workgroup of several rows has no barrier
    const int H = a.H;

    const E *r_row = static_cast<const E *>(a.residual) + row * a.ldr;
    const E *y_row = static_cast<const E *>(a.y) + row * a.ldy;
    const E *g_row = static_cast<const E *>(a.gate) + row * a.ldg;
    const bool has_y = a.y != nullptr, gate_rows = a.gate && a.ldg != 0, gate_vector = a.gate && a.ldg == 0;

    uint4 ru[C], yu[C], gu[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int k = (c * TPR + t) * V;
        yu[c] = gu[c] = make_uint4(0, 0, 0, 0);
        if (has_y) yu[c] = load_chunk<D, WHOLE, true>(y_row, k, H);
        ru[c] = load_chunk<D, WHOLE, true>(r_row, k, H);
        if (gate_rows) gu[c] = load_chunk<D, WHOLE, true>(g_row, k, H);
    }
    // the vectors: with the row where there is room for them
    constexpr bool kEarly = C <= 2 && TPR < 1024;
    const float *const vectors[3] = {a.weight, a.post ? a.post_weight : nullptr,
                                     gate_vector ? static_cast<const float *>(a.gate) : nullptr};
    float kept[kEarly ? 3 : 1][C][V];
    if constexpr (kEarly) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
            for (int c = 0; c < C; ++c) load_vector<D, WHOLE>(vectors[i], (c * TPR + t) * V, H, 1.0f, kept[i][c]);
    }
    auto vector = [&](int i, int c, float (&f)[V]) {
        if constexpr (kEarly) {
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] = kept[i][c][e];
        } else {
            load_vector<D, WHOLE>(vectors[i], (c * TPR + t) * V, H, 1.0f, f);
        }
    };
    // (the elements behind the row's end are 0: r, y and gate are cleared there)
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int k = (c * TPR + t) * V;
        yu[c] = settle<D, WHOLE>(yu[c], k, H);
        ru[c] = settle<D, WHOLE>(ru[c], k, H);
        if (gate_rows) gu[c] = settle<D, WHOLE>(gu[c], k, H);
    }
    float v[C][V];  // the new residual, then the output
    float sum[1] = {0.0f};
    if (has_y) {
        float inv = 1.0f;
        if (a.post) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float y[V];
                widen_chunk<D>(yu[c], y);
#pragma unroll
                for (int e = 0; e < V; ++e) sum[0] = __builtin_fmaf(y[e], y[e], sum[0]);
            }
            row_sums<TPR>(sum, red[0]);
            inv = 1.0f / __builtin_sqrtf(sum[0] / (float)H + a.eps);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = (c * TPR + t) * V;
            if (k >= H) {
#pragma unroll
                for (int e = 0; e < V; ++e) v[c][e] = 0.0f;
                continue;
            }
            float r[V], f[V], pw[V];
            widen_chunk<D>(yu[c], v[c]);
            widen_chunk<D>(ru[c], r);
            vector(1, c, pw);
            if (gate_rows) widen_chunk<D>(gu[c], f);
            else vector(2, c, f);
#pragma unroll
            for (int e = 0; e < V; ++e) v[c][e] = __builtin_fmaf(a.scale * f[e], v[c][e] * inv * pw[e], r[e]);
            store_chunk<D, WHOLE>(static_cast<E *>(a.new_residual) + row * H, k, H, narrow_chunk<D>(v[c]));
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) widen_chunk<D>(ru[c], v[c]);
    }

    sum[0] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < V; ++e) sum[0] = __builtin_fmaf(v[c][e], v[c][e], sum[0]);
    row_sums<TPR>(sum, red[1]);
    const float inv = 1.0f / __builtin_sqrtf(sum[0] / (float)H + a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int k = (c * TPR + t) * V;
        if (k >= H) continue;
        float w[V];
        vector(0, c, w);
#pragma unroll
        for (int e = 0; e < V; ++e) v[c][e] = v[c][e] * inv * w[e];
        if constexpr (O == kSame)
            store_chunk<D, WHOLE>(static_cast<E *>(a.out) + row * H, k, H, narrow_chunk<D>(v[c]));
    }
    if constexpr (O == kInt8) {
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < V; ++e) top = max(top, __float_as_uint(v[c][e]) & 0x7FFFFFFFu);
        top = across_row<TPR>(top, [](uint32_t x, uint32_t y) { return max(x, y); });
        if constexpr (TPR > kWave) {
            if (threadIdx.x % kWave == 0) red_max[threadIdx.x / kWave] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < TPR / kWave; ++w) top = max(top, red_max[w]);
        }
        const w8a8::RowScale rs = w8a8::row_scale(__uint_as_float(top));
        int8_t *q = static_cast<int8_t *>(a.out) + row * H;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = (c * TPR + t) * V;
            if (k >= H) continue;
            float e8[8] = {};
#pragma unroll
            for (int e = 0; e < V; ++e) e8[e] = v[c][e];
            const uint2 b = w8a8::quantize8(e8, rs);
            if constexpr (V == 8) *reinterpret_cast<uint2 *>(q + k) = b;
            else *reinterpret_cast<uint32_t *>(q + k) = b.x;
        }
        if (t == 0) static_cast<float *>(a.out_scale)[row] = rs.s;
    }
    if constexpr (O == kMxfp4) {
        uint8_t *q = static_cast<uint8_t *>(a.out) + row * (H / 2);
        uint8_t *sc = static_cast<uint8_t *>(a.out_scale);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            // up to the scales' padding behind the row's last block: its codes are 0
            const int k = (c * TPR + t) * V;
            if (c * TPR * V >= H) continue;
            uint32_t codes;
            const uint32_t code = mx_block<V>(v[c], codes);
            if (k < H) {
                if constexpr (V == 8) *reinterpret_cast<uint32_t *>(q + k / 2) = codes;
                else *reinterpret_cast<uint16_t *>(q + k / 2) = (uint16_t)codes;
            }
            if (k % 32 == 0 && k < ((H + 255) & ~255))
                sc[((int64_t)(k / 256) * a.T + row) * 8 + k / 32 % 8] = (uint8_t)code;
        }
    }
}

template <Dtype D, Out O, int TPR, int C>
hipError_t launch(const Forward &a, hipStream_t stream) {
    constexpr int kThreads = TPR <= kWave ? 256 : TPR, kRows = kThreads / TPR;
    const dim3 grid((unsigned)((a.T + kRows - 1) / kRows)), block(kThreads);
    // (quantized rows have whole chunks by their rules on widths)
    if (O != kSame || a.H % kPer<D> == 0) norm_kernel<D, O, TPR, C, true><<<grid, block, 0, stream>>>(a);
    else norm_kernel<D, O, TPR, C, O != kSame><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

// Up to so many rows, a row's latency counts more than the rows at once.
constexpr int kFewRows = 512;

template <Dtype D, Out O>
hipError_t launch_row(const Forward &a, hipStream_t stream) {
    constexpr int V = kPer<D>;
    const int chunks = (a.H + V - 1) / V;
    // a chunk or two per thread; few rows over more threads each (one step of 16 rows of 4096:
    // 5.3 -> 4.2 us)
    if constexpr (O != kMxfp4) {   // (whose scales are padded to 256 elements)
        if (chunks <= 16) return launch<D, O, 16, 1>(a, stream);
    }
    if (chunks <= 64) return launch<D, O, 64, 1>(a, stream);
    if (chunks <= 256 && a.T <= kFewRows) return launch<D, O, 256, 1>(a, stream);
    if (chunks <= 128) return launch<D, O, 64, 2>(a, stream);
    if (chunks <= 256) return launch<D, O, 128, 2>(a, stream);
    if (chunks <= 512) {
        if (a.T <= kFewRows) return launch<D, O, 512, 1>(a, stream);
        return launch<D, O, 256, 2>(a, stream);
    }
    if (chunks <= 1024) return launch<D, O, 512, 2>(a, stream);
    if constexpr (D == kF32) {
        if (chunks > 2048) return launch<D, O, 1024, 4>(a, stream);
    }
    return launch<D, O, 1024, 2>(a, stream);
}

template <Dtype D>
hipError_t launch_out(const Forward &a, int out, hipStream_t stream) {
    switch (out) {
        case kSame: return launch_row<D, kSame>(a, stream);
        case kInt8: return launch_row<D, kInt8>(a, stream);
        default: return launch_row<D, kMxfp4>(a, stream);
    }
}

}  // namespace

hipError_t launch_forward(const Forward &a, int dtype, int out, hipStream_t stream) {
    switch (dtype) {
        case kBf16: return launch_out<kBf16>(a, out, stream);
        case kF16: return launch_out<kF16>(a, out, stream);
        default: return launch_out<kF32>(a, out, stream);
    }
}

}  // namespace block
