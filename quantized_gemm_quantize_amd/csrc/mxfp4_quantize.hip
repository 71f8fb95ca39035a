// MXFP4 rows: quantization at run time and back.
//
// The quantization itself is in mxfp4_rows.hpp (the expert layer runs it beside
// its sort). Both kernels are bound by HBM; measured at 16448 x 5120 (f32, 382
// MB each way): quantize 70 us, back 55 us (129 with 32 bytes per lane, whose
// stores are not contiguous).
#include <algorithm>

#include "launch.hpp"
#include "mxfp4_rows.hpp"

namespace mxfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kHalves = kThreads / 32;  // 32-lane halves per workgroup

template <Dtype D, int U>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const char *__restrict__ x, int64_t ldx,
                                                            int64_t M, int K, int KB,
                                                            uint8_t *__restrict__ codes,
                                                            uint8_t *__restrict__ scales) {
    quantize_steps<D, U, kThreads>(blockIdx.x, x, ldx, M, K, KB, codes, scales);
}

// 16 bytes of values per lane and store (4 or 8 elements), a wavefront's stores
// contiguous; U stores per thread, their codes loaded together.
template <Dtype D, int U>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ scales,
                                                              int64_t M, int K, int KB,
                                                              void *__restrict__ out) {
    constexpr int V = D == kF32 ? 4 : 8;         // elements per lane and store
    constexpr int LANES = kStep / V;             // lanes per 256-element step
    constexpr int GROUPS = kThreads / LANES;
    const int group = threadIdx.x / LANES, i = threadIdx.x % LANES;
    const int64_t first = (int64_t)blockIdx.x * (GROUPS * U);
    const int64_t row0 = first / KB;
    const int step0 = (int)(first - row0 * KB);
    uint32_t c[U], sc[U];
    int64_t row[U];
    int k[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t s = (uint32_t)(step0 + group + u * GROUPS);
        const uint32_t r = s / (uint32_t)KB;
        const int step = (int)(s - r * KB);
        row[u] = row0 + r;
        k[u] = step * kStep + V * i;
        c[u] = sc[u] = 0;
        if (row[u] < M && k[u] < K) {
            const uint8_t *p = codes + row[u] * (K / 2) + k[u] / 2;
            c[u] = V == 8 ? *reinterpret_cast<const uint32_t *>(p) : *reinterpret_cast<const uint16_t *>(p);
            sc[u] = scales[((int64_t)step * M + row[u]) * 8 + V * i / 32];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (row[u] >= M || k[u] >= K) continue;
        const float s = scale_value(sc[u]);
        float f[V];
        w8a8::v2f p;
        p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], 1.0f, 0); f[0] = p[0] * s; f[1] = p[1] * s;
        p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], 1.0f, 1); f[2] = p[0] * s; f[3] = p[1] * s;
        if constexpr (V == 8) {
            p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], 1.0f, 2); f[4] = p[0] * s; f[5] = p[1] * s;
            p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], 1.0f, 3); f[6] = p[0] * s; f[7] = p[1] * s;
        }
        const int64_t at = row[u] * K + k[u];
        if constexpr (D == kF32) {
            w8a8::store16_nt(static_cast<float *>(out) + at, __builtin_bit_cast(uint4, v4f{f[0], f[1], f[2], f[3]}));
        } else {
            uint32_t q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (D == kBf16) q[j] = w8a8::pack_bf16x2(f[2 * j], f[2 * j + 1]);
                else q[j] = __builtin_bit_cast(uint32_t, v2h{(_Float16)f[2 * j], (_Float16)f[2 * j + 1]});
            }
            w8a8::store16_nt(static_cast<uint16_t *>(out) + at, make_uint4(q[0], q[1], q[2], q[3]));
        }
    }
}

template <Dtype D>
hipError_t dequantize_type(const uint8_t *codes, const uint8_t *scales, int64_t M, int K, void *out,
                           hipStream_t stream) {
    const int KB = (K + kStep - 1) / kStep;
    constexpr int GROUPS = kThreads / (kStep / (D == kF32 ? 4 : 8));
    const int64_t steps = M * KB;
    constexpr int U = 2;
    if (steps < (int64_t)GROUPS * U * 4 * w8a8::device_cu_count())
        dequantize_kernel<D, 1><<<dim3((unsigned)((steps + GROUPS - 1) / GROUPS)), dim3(kThreads), 0, stream>>>(codes, scales, M, K, KB, out);
    else
        dequantize_kernel<D, U><<<dim3((unsigned)((steps + GROUPS * U - 1) / (GROUPS * U))), dim3(kThreads), 0, stream>>>(codes, scales, M, K, KB, out);
    return hipGetLastError();
}

template <Dtype D>
hipError_t quantize_type(const void *x, int64_t ldx, int64_t M, int K, uint8_t *codes,
                         uint8_t *scales, hipStream_t stream) {
    const int KB = (K + kStep - 1) / kStep;
    const int64_t steps = M * KB;
    const dim3 block(kThreads);
    const char *p = static_cast<const char *>(x);
    // two loads in flight per thread: one of 32-bit steps, two of 16-bit steps
    // (38400 x 1024 bf16 21.3 -> 20.3 us; 16448 x 5120 f32 70.1, 72.0 with four)
    constexpr int U = D == kF32 ? 1 : 2;
    if (steps < (int64_t)kHalves * U * 4 * w8a8::device_cu_count())
        quantize_kernel<D, 1><<<dim3((unsigned)((steps + kHalves - 1) / kHalves)), block, 0, stream>>>(p, ldx, M, K, KB, codes, scales);
    else
        quantize_kernel<D, U><<<dim3((unsigned)((steps + kHalves * U - 1) / (kHalves * U))), block, 0, stream>>>(p, ldx, M, K, KB, codes, scales);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize(const void *x, int64_t ldx, int64_t M, int K, int dtype, uint8_t *codes,
                           uint8_t *scales, hipStream_t stream) {
    switch (dtype) {
        case kBf16: return quantize_type<kBf16>(x, ldx, M, K, codes, scales, stream);
        case kF16: return quantize_type<kF16>(x, ldx, M, K, codes, scales, stream);
        default: return quantize_type<kF32>(x, ldx, M, K, codes, scales, stream);
    }
}

hipError_t launch_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t M, int K,
                             int dtype, void *out, hipStream_t stream) {
    switch (dtype) {
        case kBf16: return dequantize_type<kBf16>(codes, scales, M, K, out, stream);
        case kF16: return dequantize_type<kF16>(codes, scales, M, K, out, stream);
        default: return dequantize_type<kF32>(codes, scales, M, K, out, stream);
    }
}

}  // namespace mxfp4
