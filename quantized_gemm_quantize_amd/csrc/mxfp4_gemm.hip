// MXFP4 x MXFP4 products: a dense layer, or rows grouped by expert.
//
//   out[m, n] = sum over blocks b of 2^(ex[m,b] + ew[n,b]) * sum_{k in b} qx[m,k] qw[n,k]
//
// on gfx950's scaled MFMA, which multiplies two fp4 blocks of 32 with their
// scales and accumulates in fp32. Every 256-element step of K, lanes 0-31 of
// a wavefront take blocks 0-3 of their row and lanes 32-63 blocks 4-7, for
// both operands: the four K steps use the four bytes of one scale register.
#include "launch.hpp"
#include "mxfp4_epilogue.hpp"

namespace mxfp4 {
namespace {

constexpr int kWaves = 4;

// Each wavefront: 32 rows x 64 channels, operands straight from memory.
template <Epilogue EP>
__global__ __launch_bounds__(kWaves *kWave) void gemm_kernel(
    const uint8_t *__restrict__ xq, const uint8_t *__restrict__ xs, const uint8_t *__restrict__ wq,
    const uint8_t *__restrict__ ws, Groups g, int N, int K, int KB, Output o) {
    const Tile t = find_tile<32>(g, blockIdx.x);
    if (t.e < 0) return;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int r = lane & 31, half = lane >> 5;
    const int n0 = (blockIdx.y * kWaves + wave) * 64;
    if (n0 >= N) return;
    const int m = t.m0 + r;
    v16f acc[2] = {v16f{}, v16f{}};
    if (t.e < g.E) {
        const int64_t arow = source_row(g, min(m, t.m1 - 1));
        const uint8_t *a = xq + arow * (K / 2) + 64 * half;
        const uint8_t *as = xs + arow * 8 + 4 * half;
        const uint8_t *w[2], *wsc[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t n = min(n0 + 32 * j + r, N - 1);
            w[j] = wq + ((int64_t)t.e * N + n) * (K / 2) + 64 * half;
            wsc[j] = ws + ((int64_t)t.e * KB * N + n) * 8 + 4 * half;
        }
        for (int b = 0; b < KB; ++b) {
            const uint32_t sa = *reinterpret_cast<const uint32_t *>(as + (int64_t)b * g.T * 8);
            uint32_t sb[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                sb[j] = *reinterpret_cast<const uint32_t *>(wsc[j] + (int64_t)b * N * 8);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                // blocks past K: nothing is read, zeros multiply
                const bool in = b * kStep + 128 * half + 32 * kk < K;
                const int at = b * kStepBytes + 16 * kk;
                const v4i va = in ? *reinterpret_cast<const v4i *>(a + at) : v4i{};
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const v4i vw = in ? *reinterpret_cast<const v4i *>(w[j] + at) : v4i{};
                    acc[j] = mfma_32x32x64(kk, vw, sb[j], va, sa, acc[j]);
                }
            }
        }
    }
    const bool live = m < t.m1;
    if constexpr (EP == kSwiglu) {
        store_swiglu(acc[0], acc[1], o, m, live, n0, half, N, g.S);
    } else {
        store_tile<EP>(acc[0], o.out, m, live, n0, half, N);
        store_tile<EP>(acc[1], o.out, m, live, n0 + 32, half, N);
    }
}

}  // namespace

hipError_t launch_gemm_tiled(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq,
                             const uint8_t *ws, const Groups &g, int N, int K, int epilogue,
                             const Output &o, hipStream_t stream);

hipError_t launch_gemm(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws,
                       const Groups &g, int N, int K, int epilogue, const Output &o,
                       hipStream_t stream) {
    if (g.S > 64) return launch_gemm_tiled(xq, xs, wq, ws, g, N, K, epilogue, o, stream);
    const int KB = (K + kStep - 1) / kStep;
    const dim3 grid((unsigned)most_tiles(g.S, g.E, 32, g.offsets != nullptr),
                    (unsigned)((N + 64 * kWaves - 1) / (64 * kWaves)));
    const dim3 block(kWaves * kWave);
    switch (epilogue) {
        case kOutBf16: gemm_kernel<kOutBf16><<<grid, block, 0, stream>>>(xq, xs, wq, ws, g, N, K, KB, o); break;
        case kOutF16: gemm_kernel<kOutF16><<<grid, block, 0, stream>>>(xq, xs, wq, ws, g, N, K, KB, o); break;
        case kOutF32: gemm_kernel<kOutF32><<<grid, block, 0, stream>>>(xq, xs, wq, ws, g, N, K, KB, o); break;
        default: gemm_kernel<kSwiglu><<<grid, block, 0, stream>>>(xq, xs, wq, ws, g, N, K, KB, o);
    }
    return hipGetLastError();
}

}  // namespace mxfp4
