// 16-bit products of a few rows: the weight is streamed once.
//
//   out[m, n] = epilogue( sum_k x[m, k] w[n, k] ),  m < 16 MT
//
// Every weight byte serves 16 MT multiply-adds at most, so the time is that of reading w.
// One workgroup takes 16 channels; its WAVES wavefronts take the 128-byte pieces of K (64 k)
// in turn, wavefront v pieces v, v + WAVES, ..., and each keeps P pieces of both operands in
// flight in LDS of its own (16-byte direct-to-LDS loads in whole cache lines), so no barrier
// stands between the stream and the matrix instructions. A piece: 16 weight rows, then the 16 MT
// activation rows, of 8 chunks, chunk c of row r at slot c ^ swz(r) as in linear16_tiled.hip.
// The wavefronts' partial tiles are summed in LDS in a fixed order; a thread then finishes four
// consecutive channels of a row.
// Measured: 1 x 4096 x 4096 5.8 us (5.8 TB/s of weights), 64 x 4096 x 2048 9.0: there the rows' own
// loads are four times the weights'.
#include "activation.hpp"
#include "launch.hpp"
#include "linear16.hpp"
#include "linear16_mfma.hpp"
#include "rows.hpp"

namespace linear16 {
namespace {

using rows::kBf16;
using rows::kF16;

template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
    asm volatile("" ::: "memory");
}

struct Rows {
    const char *x, *w;
    int64_t ldx, ldw;   // bytes
    int M, N, K;
    Epilogue ep;
};

// The products of the piece in rd. (The compiler takes rd and the buffers that loads are written to for
// distinct, so that it does not wait for loads in flight here; the caller has waited for this piece.)
template <bool F16, int MT>
__device__ __forceinline__ void multiply(const uint4 *__restrict__ rd, int lane, int k_left, v4f (&acc)[MT]) {
    const int r = lane & 15, group = lane >> 4;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int c = 4 * t + group, slot = r * 8 + (c ^ swz(r));
        const bool in = 8 * c < k_left;
        const v4i w = in ? __builtin_bit_cast(v4i, rd[slot]) : v4i{};
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const v4i x = in ? __builtin_bit_cast(v4i, rd[(i + 1) * 128 + slot]) : v4i{};
            acc[i] = mfma<F16>(w, x, acc[i]);
        }
    }
}

template <bool F16, int MT, int WAVES, int P>
__global__ __launch_bounds__(WAVES *kWave) void rows_kernel(const Rows g) {
    constexpr int kPiece = 128 * (MT + 1);   // 16-byte slots
    constexpr int kLoads = 2 * (MT + 1);     // per piece
    __shared__ uint4 lds[WAVES * P * kPiece];
    static_assert(WAVES * MT * 64 <= WAVES * P * kPiece, "the partial tiles fit");
    w8a8::lds_poison(lds);
    w8a8::lds_poison_done();
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int n0 = blockIdx.x * 16;
    uint4 *const mine = lds + wave * P * kPiece;

    // load h of 16 rows: rows 8 h + lane / 8, the chunk that belongs into slot lane % 8
    const char *at[kLoads];
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
        const int row = 8 * l + lane / 8;   // in the piece
        at[l] = l < 2 ? g.w + (int64_t)min(n0 + row, g.N - 1) * g.ldw : g.x + (int64_t)min(row - 16, g.M - 1) * g.ldx;
    }
    const int row8 = lane / 8;
    const int pieces = (g.K + 63) / 64, count = (pieces - wave + WAVES - 1) / WAVES;
    auto issue = [&](int i) {
        const int k = 64 * (wave + i * WAVES);
        uint4 *to = mine + i % P * kPiece;
#pragma unroll
        for (int l = 0; l < kLoads; ++l) {
            const int c = (lane % 8) ^ swz(8 * l + row8);
            // a chunk past K is read from the row's last one, and zeroed as it is used
            const char *from = at[l] + 2 * min(k + 8 * c, g.K - 8);
            if (l < 2) __builtin_amdgcn_global_load_lds((global_void *)from, (lds_void *)(to + 64 * l), 16, 0, w8a8::kLdsLoadStream);
            else __builtin_amdgcn_global_load_lds((global_void *)from, (lds_void *)(to + 64 * l), 16, 0, 0);
        }
    };

    v4f acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = v4f{};
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (i < count) issue(i);
    for (int i = 0; i < count; ++i) {
        if (i + P - 1 < count) wait_loads<(P - 1) * kLoads>();
        else wait_loads<0>();
        multiply<F16, MT>(mine + i % P * kPiece, lane, g.K - 64 * (wave + i * WAVES), acc);
        // the piece is in registers before its buffer is filled again
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (i + P < count) issue(i + P);
    }
    __syncthreads();

    v4f *red = reinterpret_cast<v4f *>(lds);
#pragma unroll
    for (int i = 0; i < MT; ++i) red[(wave * MT + i) * kWave + lane] = acc[i];
    __syncthreads();
    constexpr auto D = F16 ? kF16 : kBf16;
    for (int q = threadIdx.x; q < MT * kWave; q += WAVES * kWave) {
        const int m = q / kWave * 16 + q % 16, n = n0 + q % kWave / 16 * 4;
        if (m >= g.M || n >= g.N) continue;
        v4f sum = red[q];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) sum += red[w * MT * kWave + q];
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = sum[e] + (g.ep.bias ? g.ep.bias[n + e] : 0.0f);
        auto store = [&](void *to) {
            uint2 u;
            u.x = (uint32_t)rows::narrow<D>(v[0]) | (uint32_t)rows::narrow<D>(v[1]) << 16;
            u.y = (uint32_t)rows::narrow<D>(v[2]) | (uint32_t)rows::narrow<D>(v[3]) << 16;
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(to) + (int64_t)m * g.N + n) = u;
        };
        if (g.ep.pre) store(g.ep.pre);
        act::activate(g.ep.act, v);
        if (g.ep.residual) {
            const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(g.ep.residual) + m * g.ep.ldr + n);
            v[0] += rows::widen<D>((uint16_t)u.x);
            v[1] += rows::widen<D>((uint16_t)(u.x >> 16));
            v[2] += rows::widen<D>((uint16_t)u.y);
            v[3] += rows::widen<D>((uint16_t)(u.y >> 16));
        }
        store(g.ep.out);
    }
}

template <bool F16, int MT, int WAVES, int P>
hipError_t launch(const Rows &g, hipStream_t stream) {
    rows_kernel<F16, MT, WAVES, P><<<dim3((unsigned)((g.N + 15) / 16)), WAVES * kWave, 0, stream>>>(g);
    return hipGetLastError();
}

template <bool F16>
hipError_t launch_type(const Rows &g, hipStream_t stream) {
    switch ((g.M + 15) / 16) {
        case 1: return launch<F16, 1, 8, 2>(g, stream);
        case 2: return launch<F16, 2, 8, 3>(g, stream);
        case 3: return launch<F16, 3, 8, 2>(g, stream);
        default: return launch<F16, 4, 8, 2>(g, stream);
    }
}

}  // namespace

hipError_t launch_rows(const void *x, int64_t ldx, int M, const void *w, int N, int K, bool f16, const Epilogue &ep,
                       hipStream_t stream) {
    const Rows g{static_cast<const char *>(x), static_cast<const char *>(w), 2 * ldx, 2 * (int64_t)K, M, N, K, ep};
    return f16 ? launch_type<true>(g, stream) : launch_type<false>(g, stream);
}

}  // namespace linear16
