// C ABI of libw8a8.so: argument validation, then one launch on the caller's
// stream. Declarations and argument contracts are in include/w8a8.h.
//
// Every check runs on the host before any HIP call, so a rejected call
// touches no device state. Failures return a nonzero status, as the pages'
// TensorRT plugin does with its library status (Paddle sparse_fc PR #41770,
// spmm_plugin.cu enqueue hunk).
#include "w8a8.h"

#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstring>

#include "activation.hpp"
#include "common.hpp"
#include "launch.hpp"
#include "linear16.hpp"
#include "mxfp4_epilogue.hpp"
#include "mxfp4_form.hpp"
#include "norm.hpp"

namespace {

thread_local int g_last_hip_error = 0;

bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// A C caller may pass any int for an enum parameter, but in C++ reading an
// enum object whose value lies outside its enumerators' range is undefined:
// selectors are read as the int they are, then validated.
template <typename E>
int selector(const E *e) {
    static_assert(sizeof(E) == sizeof(int), "C enums are int-sized here");
    int v;
    std::memcpy(&v, e, sizeof v);
    return v;
}

w8a8_status hip_status(hipError_t e) {
    if (e == hipSuccess) return W8A8_OK;
    g_last_hip_error = static_cast<int>(e);
    return W8A8_ERR_HIP;
}

// K checks shared by every entry: positive multiple of 16, int32-safe.
w8a8_status check_k(int64_t K) {
    if (K <= 0 || K % 16 != 0) return W8A8_ERR_SHAPE;
    if (K > W8A8_MAX_K) return W8A8_ERR_K_OVERFLOW;
    return W8A8_OK;
}

// Sizes the kernels index with 32-bit integers.
bool too_big(int64_t M, int64_t N) { return M > INT_MAX / 2 || N > INT_MAX / 2; }

// Whether a dense product's launch holds fewer than 2^32 threads: up to 64 rows, 512 of them (1024 for a long K) for 16
// channels; above, 256 for a tile of 256 x 128 (smaller tiles are taken for a few hundred of them only).
bool dense_launch(int64_t M, int64_t N, int64_t K) {
    return M <= 64 ? w8a8::grid_fits(N / 16, K > 4096 ? 1024 : 512)
                   : w8a8::grid_fits((M + 255) / 256 * ((N + 127) / 128), 256);
}

template <typename T>
w8a8_status quantize_entry(const T *x, int64_t M, int64_t K, int8_t *xq, float *x_scale,
                           void *stream,
                           hipError_t (*launch)(const T *, int64_t, int, int8_t *, float *,
                                                hipStream_t)) {
    if (M < 0) return W8A8_ERR_SHAPE;
    if (w8a8_status s = check_k(K)) return s;
    if (M == 0) return W8A8_OK;
    if (M > INT_MAX) return W8A8_ERR_SHAPE;  // grid.x: at least one row per workgroup
    if (!x || !xq || !x_scale) return W8A8_ERR_NULL;
    if (misaligned(x) || misaligned(xq) || misaligned(x_scale)) return W8A8_ERR_ALIGN;
    return hip_status(launch(x, M, (int)K, xq, x_scale, static_cast<hipStream_t>(stream)));
}

}  // namespace

namespace w8a8 {

int device_cu_count() {
    static int cus[64] = {};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    if (cus[dev] == 0) {
        int n = 0;
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
            n <= 0)
            n = 256;
        cus[dev] = n;
    }
    return cus[dev];
}

}  // namespace w8a8

extern "C" {

w8a8_status w8a8_quantize_rows(const void *x_bf16, int64_t M, int64_t K, int8_t *xq,
                               float *x_scale, void *stream) {
    return quantize_entry<uint16_t>(static_cast<const uint16_t *>(x_bf16), M, K, xq, x_scale,
                                    stream, w8a8::launch_quantize_rows_bf16);
}

w8a8_status w8a8_quantize_rows_f32(const float *x, int64_t M, int64_t K, int8_t *xq,
                                   float *x_scale, void *stream) {
    return quantize_entry<float>(x, M, K, xq, x_scale, stream, w8a8::launch_quantize_rows_f32);
}

w8a8_status w8a8_gemm(const int8_t *xq, const float *x_scale, int64_t M, const int8_t *wq,
                      const float *w_scale, int64_t N, int64_t K, void *out,
                      w8a8_out_dtype out_dtype, void *stream) {
    if (M < 0 || N <= 0 || N % 16 != 0 || too_big(M, N)) return W8A8_ERR_SHAPE;
    if (w8a8_status s = check_k(K)) return s;
    const int od = selector(&out_dtype);
    if (od != W8A8_OUT_BF16 && od != W8A8_OUT_I32) return W8A8_ERR_DTYPE;
    if ((M + 127) / 128 > INT_MAX / ((N + 127) / 128)) return W8A8_ERR_SHAPE;  // grid.x
    if (M == 0) return W8A8_OK;
    if (!dense_launch(M, N, K)) return W8A8_ERR_SHAPE;
    if (!xq || !x_scale || !wq || !w_scale || !out) return W8A8_ERR_NULL;
    if (misaligned(xq) || misaligned(x_scale) || misaligned(wq) || misaligned(w_scale) ||
        misaligned(out))
        return W8A8_ERR_ALIGN;
    return hip_status(w8a8::launch_gemm(xq, x_scale, (int)M, wq, w_scale, (int)N, (int)K, out,
                                        od == W8A8_OUT_I32,
                                        static_cast<hipStream_t>(stream)));
}

w8a8_status w8a8_gemm_addmm(const int8_t *xq, const float *x_scale, int64_t M, const int8_t *wq,
                            const float *w_scale, int64_t N, int64_t K, const float *bias,
                            float alpha, float beta, void *out, void *stream) {
    if (M < 0 || N <= 0 || N % 16 != 0 || too_big(M, N)) return W8A8_ERR_SHAPE;
    if (w8a8_status s = check_k(K)) return s;
    if (!std::isfinite(alpha) || !std::isfinite(beta)) return W8A8_ERR_VALUE;
    if ((M + 127) / 128 > INT_MAX / ((N + 127) / 128)) return W8A8_ERR_SHAPE;  // grid.x
    if (M == 0) return W8A8_OK;
    if (!dense_launch(M, N, K)) return W8A8_ERR_SHAPE;
    if (!xq || !x_scale || !wq || !w_scale || !out) return W8A8_ERR_NULL;
    if (!bias && beta != 0.0f) return W8A8_ERR_NULL;
    if (misaligned(xq) || misaligned(x_scale) || misaligned(wq) || misaligned(w_scale) ||
        misaligned(out) || (bias && misaligned(bias)))
        return W8A8_ERR_ALIGN;
    const w8a8::Addmm am{bias, alpha, beta};
    return hip_status(w8a8::launch_gemm(xq, x_scale, (int)M, wq, w_scale, (int)N, (int)K, out,
                                        false, static_cast<hipStream_t>(stream), &am));
}

w8a8_status w8a8_fused_linear(const void *x_bf16, int64_t M, int64_t K, const int8_t *wq,
                              const float *w_scale, int64_t N, const float *bias, float alpha,
                              float beta, void *out, void *stream) {
    if (M < 0 || M > W8A8_FUSED_MAX_M || N <= 0 || N % 16 != 0 || too_big(M, N))
        return W8A8_ERR_SHAPE;
    if (w8a8_status s = check_k(K)) return s;
    if (!std::isfinite(alpha) || !std::isfinite(beta)) return W8A8_ERR_VALUE;
    if (M == 0) return W8A8_OK;
    if (!x_bf16 || !wq || !w_scale || !out) return W8A8_ERR_NULL;
    if (!bias && beta != 0.0f) return W8A8_ERR_NULL;
    if (misaligned(x_bf16) || misaligned(wq) || misaligned(w_scale) || misaligned(out) ||
        (bias && misaligned(bias)))
        return W8A8_ERR_ALIGN;
    const w8a8::Addmm am{bias, alpha, beta};
    return hip_status(w8a8::launch_linear_decode(static_cast<const uint16_t *>(x_bf16), (int)M, wq,
                                                 w_scale, (int)N, (int)K, out,
                                                 static_cast<hipStream_t>(stream), am));
}

w8a8_status w8a8_bsr_gemm(const int8_t *xq, const float *x_scale, int64_t M, int64_t K,
                          const int32_t *crow, const int32_t *col, const int8_t *values,
                          int64_t nnzb, int64_t bs, const float *w_scale, int64_t N, void *out,
                          w8a8_out_dtype out_dtype, void *stream) {
    if (bs != 64) return W8A8_ERR_BLOCKSIZE;
    if (M < 0 || N <= 0 || N % bs != 0 || K % bs != 0 || nnzb < 0 || too_big(M, N))
        return W8A8_ERR_SHAPE;
    if (w8a8_status s = check_k(K)) return s;
    if (nnzb > (N / bs) * (K / bs)) return W8A8_ERR_SHAPE;
    const int od = selector(&out_dtype);
    if (od != W8A8_OUT_BF16 && od != W8A8_OUT_I32) return W8A8_ERR_DTYPE;
    if ((M + 127) / 128 > INT_MAX / (N / bs)) return W8A8_ERR_SHAPE;  // grid.x
    if (M == 0) return W8A8_OK;
    if (!xq || !x_scale || !crow || !w_scale || !out) return W8A8_ERR_NULL;
    if (nnzb > 0 && (!col || !values)) return W8A8_ERR_NULL;
    if (misaligned(xq) || misaligned(x_scale) || misaligned(crow) || misaligned(w_scale) ||
        misaligned(out) || (nnzb > 0 && (misaligned(col) || misaligned(values))))
        return W8A8_ERR_ALIGN;
    return hip_status(w8a8::launch_bsr_gemm(xq, x_scale, (int)M, (int)K, crow, col, values,
                                            (int)nnzb, w_scale, (int)N, out,
                                            od == W8A8_OUT_I32,
                                            static_cast<hipStream_t>(stream)));
}

w8a8_status w8a8_bsr_gemm_addmm(const int8_t *xq, const float *x_scale, int64_t M, int64_t K,
                                const int32_t *crow, const int32_t *col, const int8_t *values,
                                int64_t nnzb, int64_t bs, const float *w_scale, int64_t N,
                                const float *bias, float alpha, float beta, void *out,
                                void *stream) {
    if (bs != 64) return W8A8_ERR_BLOCKSIZE;
    if (M < 0 || N <= 0 || N % bs != 0 || K % bs != 0 || nnzb < 0 || too_big(M, N))
        return W8A8_ERR_SHAPE;
    if (w8a8_status s = check_k(K)) return s;
    if (nnzb > (N / bs) * (K / bs)) return W8A8_ERR_SHAPE;
    if (!std::isfinite(alpha) || !std::isfinite(beta)) return W8A8_ERR_VALUE;
    if ((M + 127) / 128 > INT_MAX / (N / bs)) return W8A8_ERR_SHAPE;  // grid.x
    if (M == 0) return W8A8_OK;
    if (!xq || !x_scale || !crow || !w_scale || !out) return W8A8_ERR_NULL;
    if (nnzb > 0 && (!col || !values)) return W8A8_ERR_NULL;
    if (!bias && beta != 0.0f) return W8A8_ERR_NULL;
    if (misaligned(xq) || misaligned(x_scale) || misaligned(crow) || misaligned(w_scale) ||
        misaligned(out) || (nnzb > 0 && (misaligned(col) || misaligned(values))) ||
        (bias && misaligned(bias)))
        return W8A8_ERR_ALIGN;
    const w8a8::Addmm am{bias, alpha, beta};
    return hip_status(w8a8::launch_bsr_gemm(xq, x_scale, (int)M, (int)K, crow, col, values,
                                            (int)nnzb, w_scale, (int)N, out, false,
                                            static_cast<hipStream_t>(stream), &am));
}

w8a8_status w8a8_compress24(const int8_t *wq, int64_t N, int64_t K, int8_t *values,
                            uint32_t *meta, void *stream) {
    if (N < 0 || K <= 0 || K % 128 != 0 || N > INT_MAX / 2 || K > INT_MAX / 2) return W8A8_ERR_SHAPE;
    if (N == 0) return W8A8_OK;
    if (N * (K / 32) > (int64_t)UINT_MAX * 256 / 2) return W8A8_ERR_SHAPE;  // grid.x
    if (!wq || !values || !meta) return W8A8_ERR_NULL;
    if (misaligned(wq) || misaligned(values) || misaligned(meta)) return W8A8_ERR_ALIGN;
    return hip_status(w8a8::launch_compress24(wq, (int)N, (int)K, values, meta,
                                              static_cast<hipStream_t>(stream)));
}

w8a8_status w8a8_sparse24_gemm(const int8_t *xq, const float *x_scale, int64_t M,
                               const int8_t *values, const uint32_t *meta, const float *w_scale,
                               int64_t N, int64_t K, void *out, w8a8_out_dtype out_dtype,
                               void *stream) {
    if (M < 0 || N <= 0 || N % 16 != 0 || K % 128 != 0 || too_big(M, N)) return W8A8_ERR_SHAPE;
    if (w8a8_status s = check_k(K)) return s;
    const int od = selector(&out_dtype);
    if (od != W8A8_OUT_BF16 && od != W8A8_OUT_I32) return W8A8_ERR_DTYPE;
    if ((M + 127) / 128 > INT_MAX / ((N + 255) / 256)) return W8A8_ERR_SHAPE;  // grid.x
    if (M == 0) return W8A8_OK;
    if (!xq || !x_scale || !values || !meta || !w_scale || !out) return W8A8_ERR_NULL;
    if (misaligned(xq) || misaligned(x_scale) || misaligned(values) || misaligned(meta) ||
        misaligned(w_scale) || misaligned(out))
        return W8A8_ERR_ALIGN;
    return hip_status(w8a8::launch_sparse24_gemm(xq, x_scale, (int)M, values, meta, w_scale,
                                                 (int)N, (int)K, out, od == W8A8_OUT_I32,
                                                 static_cast<hipStream_t>(stream)));
}

// W4A16 shape rules shared by both entry points.
static w8a8_status w4a16_shape(int64_t N, int64_t K, int64_t G) {
    if (N <= 0 || N % 16 != 0 || K <= 0 || K % 128 != 0 || G <= 0 || G % 32 != 0 || K % G != 0 ||
        N > INT_MAX / 2 || K > INT_MAX / 2 || N * K / 8 > (int64_t)UINT_MAX * 256 / 2)
        return W8A8_ERR_SHAPE;
    return W8A8_OK;
}

static bool misaligned2(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 1u) != 0; }

w8a8_status w4a16_dequant(const uint8_t *wq4, const void *scales, const void *zeros, int64_t N,
                          int64_t K, int64_t group_size, w4a16_codes codes, w4a16_dtype dtype,
                          void *w, void *stream) {
    if (w8a8_status s = w4a16_shape(N, K, group_size)) return s;
    const int cs = selector(&codes), dt = selector(&dtype);
    if (cs != W4A16_CODES_U4 && cs != W4A16_CODES_S4) return W8A8_ERR_DTYPE;
    if (dt != W4A16_BF16 && dt != W4A16_F16) return W8A8_ERR_DTYPE;
    if (!wq4 || !scales || !zeros || !w) return W8A8_ERR_NULL;
    if (misaligned(wq4) || misaligned(w) || misaligned2(scales) || misaligned2(zeros))
        return W8A8_ERR_ALIGN;
    return hip_status(w4a16::launch_dequant(wq4, static_cast<const uint16_t *>(scales),
                                            static_cast<const uint16_t *>(zeros), (int)N, (int)K,
                                            (int)group_size, cs == W4A16_CODES_S4,
                                            dt == W4A16_F16, static_cast<uint16_t *>(w),
                                            static_cast<hipStream_t>(stream)));
}

w8a8_status w4a16_gemm(const void *x, int64_t M, const uint8_t *wq4, const void *scales,
                       const void *zeros, int64_t N, int64_t K, int64_t group_size,
                       w4a16_codes codes, w4a16_dtype dtype, void *out, void *stream) {
    if (M < 0 || M > INT_MAX / 2) return W8A8_ERR_SHAPE;
    if (w8a8_status s = w4a16_shape(N, K, group_size)) return s;
    const int cs = selector(&codes), dt = selector(&dtype);
    if (cs != W4A16_CODES_U4 && cs != W4A16_CODES_S4) return W8A8_ERR_DTYPE;
    if (dt != W4A16_BF16 && dt != W4A16_F16) return W8A8_ERR_DTYPE;
    if ((M + 63) / 64 > INT_MAX / ((N + 63) / 64)) return W8A8_ERR_SHAPE;  // grid.x
    if (M == 0) return W8A8_OK;
    if (!x || !wq4 || !scales || !zeros || !out) return W8A8_ERR_NULL;
    if (misaligned(x) || misaligned(wq4) || misaligned(out) || misaligned2(scales) ||
        misaligned2(zeros))
        return W8A8_ERR_ALIGN;
    return hip_status(w4a16::launch_gemm(static_cast<const uint16_t *>(x), (int)M, wq4,
                                         static_cast<const uint16_t *>(scales),
                                         static_cast<const uint16_t *>(zeros), (int)N, (int)K,
                                         (int)group_size, cs == W4A16_CODES_S4,
                                         dt == W4A16_F16, static_cast<uint16_t *>(out),
                                         static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------- MXFP4

static bool mx_dtype_ok(int d) { return d == MXFP4_BF16 || d == MXFP4_F16 || d == MXFP4_F32; }

static int64_t dtype_size(int d) { return d == MXFP4_F32 ? 4 : 2; }

// K and rows that the MXFP4 kernels index with 32-bit step counts.
static w8a8_status mx_shape(int64_t rows, int64_t K) {
    if (rows < 0 || rows > INT_MAX / 2 || K <= 0 || K % 32 != 0 || K > MXFP4_MAX_K)
        return W8A8_ERR_SHAPE;
    // 32 threads per 256 elements, 8 of them to a workgroup
    if (rows * ((K + 255) / 256) > (1 << 27) - 8) return W8A8_ERR_SHAPE;
    return W8A8_OK;
}

static w8a8_status mx_weight(int64_t N, int64_t K) {
    if (N <= 0 || N % 16 != 0) return W8A8_ERR_SHAPE;
    return mx_shape(N, K);
}

// Outputs of a product: at most 2^36 (the kernels count tiles in 32 bits, and a dense
// product's workgroups are then within a grid's threads).
static w8a8_status mx_out(int64_t rows, int64_t N) {
    return rows > 0 && N > ((int64_t)1 << 36) / rows ? W8A8_ERR_SHAPE : W8A8_OK;
}

// Activation rows that are read through row_token lie within 32-bit offsets.
static w8a8_status mx_tokens(int64_t T, int64_t K) {
    return T * (K / 2) > (int64_t)UINT_MAX ? W8A8_ERR_SHAPE : W8A8_OK;
}

static int64_t align256(int64_t bytes) { return (bytes + 255) / 256 * 256; }
static int64_t mx_codes(int64_t rows, int64_t K) { return align256(rows * (K / 2)); }
static int64_t mx_scales(int64_t rows, int64_t K) { return align256((K + 255) / 256 * rows * 8); }

w8a8_status mxfp4_quantize_rows(const void *x, int64_t ldx, int64_t M, int64_t K,
                                mxfp4_dtype dtype, uint8_t *codes, uint8_t *scales, void *stream) {
    if (w8a8_status s = mx_shape(M, K)) return s;
    if (ldx < K || ldx > INT_MAX) return W8A8_ERR_SHAPE;
    const int dt = selector(&dtype);
    if (!mx_dtype_ok(dt)) return W8A8_ERR_DTYPE;
    if (M == 0) return W8A8_OK;
    if (!x || !codes || !scales) return W8A8_ERR_NULL;
    if (misaligned(x) || misaligned(codes) || misaligned(scales) || ldx * dtype_size(dt) % 16 != 0)
        return W8A8_ERR_ALIGN;
    return hip_status(mxfp4::launch_quantize(x, ldx, M, (int)K, dt, codes, scales,
                                             static_cast<hipStream_t>(stream)));
}

w8a8_status mxfp4_dequantize_rows(const uint8_t *codes, const uint8_t *scales, int64_t M,
                                  int64_t K, mxfp4_dtype dtype, void *out, void *stream) {
    if (w8a8_status s = mx_shape(M, K)) return s;
    const int dt = selector(&dtype);
    if (!mx_dtype_ok(dt)) return W8A8_ERR_DTYPE;
    if (M == 0) return W8A8_OK;
    if (!codes || !scales || !out) return W8A8_ERR_NULL;
    if (misaligned(codes) || misaligned(scales) || misaligned(out)) return W8A8_ERR_ALIGN;
    return hip_status(mxfp4::launch_dequantize(codes, scales, M, (int)K, dt, out,
                                               static_cast<hipStream_t>(stream)));
}

w8a8_status mxfp4_gemm(const uint8_t *xq, const uint8_t *xs, int64_t M, const uint8_t *wq,
                       const uint8_t *ws, int64_t N, int64_t K, mxfp4_dtype dtype, void *out,
                       void *stream) {
    if (w8a8_status s = mx_shape(M, K)) return s;
    if (w8a8_status s = mx_weight(N, K)) return s;
    if (w8a8_status s = mx_out(M, N)) return s;
    const int dt = selector(&dtype);
    if (!mx_dtype_ok(dt)) return W8A8_ERR_DTYPE;
    if (M == 0) return W8A8_OK;
    if (!xq || !xs || !wq || !ws || !out) return W8A8_ERR_NULL;
    if (misaligned(xq) || misaligned(xs) || misaligned(wq) || misaligned(ws) || misaligned(out))
        return W8A8_ERR_ALIGN;
    const mxfp4::Groups g{nullptr, nullptr, 1, (int)M, (int)M};
    return hip_status(mxfp4::launch_gemm(xq, xs, wq, ws, g, (int)N, (int)K, dt,
                                         mxfp4::Output{out, nullptr, nullptr},
                                         static_cast<hipStream_t>(stream)));
}

int64_t mxfp4_linear_workspace(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || mx_shape(M, K) != W8A8_OK || mxfp4::single_launch_linear(M, N)) return 0;
    return mx_codes(M, K) + mx_scales(M, K);
}

w8a8_status mxfp4_linear(const void *x, int64_t ldx, mxfp4_dtype x_dtype, int64_t M,
                         const uint8_t *wq, const uint8_t *ws, int64_t N, int64_t K,
                         mxfp4_dtype out_dtype, void *out, void *workspace,
                         int64_t workspace_bytes, void *stream) {
    if (w8a8_status s = mx_shape(M, K)) return s;
    if (w8a8_status s = mx_weight(N, K)) return s;
    if (w8a8_status s = mx_out(M, N)) return s;
    const int xd = selector(&x_dtype), od = selector(&out_dtype);
    if (!mx_dtype_ok(xd) || !mx_dtype_ok(od)) return W8A8_ERR_DTYPE;
    if (ldx < K || ldx > INT_MAX || workspace_bytes < mxfp4_linear_workspace(M, N, K))
        return W8A8_ERR_SHAPE;
    if (M == 0) return W8A8_OK;
    const bool fused = mxfp4::single_launch_linear(M, N);
    if (!x || !wq || !ws || !out || (!fused && !workspace)) return W8A8_ERR_NULL;
    if (misaligned(x) || misaligned(wq) || misaligned(ws) || misaligned(out) ||
        misaligned(workspace) || ldx * dtype_size(xd) % 16 != 0)
        return W8A8_ERR_ALIGN;
    if (fused)
        return hip_status(mxfp4::launch_linear_decode(x, ldx, xd, (int)M, wq, ws, (int)N, (int)K, od,
                                                      out, static_cast<hipStream_t>(stream)));
    uint8_t *codes = static_cast<uint8_t *>(workspace), *scales = codes + mx_codes(M, K);
    if (w8a8_status s = mxfp4_quantize_rows(x, ldx, M, K, x_dtype, codes, scales, stream)) return s;
    return mxfp4_gemm(codes, scales, M, wq, ws, N, K, out_dtype, out, stream);
}

// ---------------------------------------------------------------- experts

// T, top and E of a routing plan.
static w8a8_status moe_shape(int64_t T, int64_t top) {
    if (T < 0 || top <= 0 || T >= (1 << 24) || top >= (1 << 30) || T * top >= (1 << 30))
        return W8A8_ERR_SHAPE;  // a workgroup of 256 threads per token
    return W8A8_OK;
}

static bool odd(const void *p, int64_t size) {
    return reinterpret_cast<uintptr_t>(p) % (uintptr_t)size != 0;
}

int64_t moe_sort_workspace(int64_t slots, int64_t E) {
    return slots <= 0 || slots >= (1 << 30) || E <= 0 || E > MOE_MAX_EXPERTS
               ? 0 : moe::sort_workspace(slots, E);
}

w8a8_status moe_sort(const void *expert_ids, int ids_bits, int64_t T, int64_t top, int64_t E,
                     int32_t *offsets, int32_t *slot_pos, int32_t *row_token, void *workspace,
                     int64_t workspace_bytes, void *stream) {
    if (w8a8_status s = moe_shape(T, top)) return s;
    if (E <= 0 || E > MOE_MAX_EXPERTS) return W8A8_ERR_SHAPE;
    if (ids_bits != 32 && ids_bits != 64) return W8A8_ERR_DTYPE;
    const int64_t need = moe_sort_workspace(T * top, E);
    if (workspace_bytes < need) return W8A8_ERR_SHAPE;
    if (!offsets || (need > 0 && !workspace)) return W8A8_ERR_NULL;
    if (T > 0 && (!expert_ids || !slot_pos || !row_token)) return W8A8_ERR_NULL;
    if (odd(expert_ids, ids_bits / 8) || odd(offsets, 4) || odd(slot_pos, 4) || odd(row_token, 4) ||
        odd(workspace, 4))
        return W8A8_ERR_ALIGN;
    return hip_status(moe::launch_sort(expert_ids, ids_bits == 64, T * top, (int)top, (int)E,
                                       offsets, slot_pos, row_token, workspace,
                                       static_cast<hipStream_t>(stream)));
}

// Shapes that the row kernels take: T workgroups along x, H in segments.
static w8a8_status moe_rows(int64_t T, int64_t top, int64_t H, int64_t ld) {
    if (w8a8_status s = moe_shape(T, top)) return s;
    if (H <= 0 || H > (1 << 23) || ld < H || ld > INT_MAX) return W8A8_ERR_SHAPE;
    return W8A8_OK;
}

w8a8_status moe_gather(const void *x, int64_t ldx, const int32_t *slot_pos, int64_t T, int64_t top,
                       int64_t H, mxfp4_dtype dtype, void *rows, void *stream) {
    if (w8a8_status s = moe_rows(T, top, H, ldx)) return s;
    const int dt = selector(&dtype);
    if (!mx_dtype_ok(dt)) return W8A8_ERR_DTYPE;
    if (T == 0) return W8A8_OK;
    if (!x || !slot_pos || !rows) return W8A8_ERR_NULL;
    const int64_t size = dtype_size(dt);
    if (odd(x, size) || odd(rows, size) || odd(slot_pos, 4)) return W8A8_ERR_ALIGN;
    return hip_status(moe::launch_gather(x, ldx, slot_pos, T, (int)top, (int)H, dt, rows,
                                         static_cast<hipStream_t>(stream)));
}

// combine, and (weights null) the gather's gradient
static w8a8_status combine_entry(const void *rows, const int32_t *slot_pos, const float *weights,
                                 bool weighted, int64_t T, int64_t top, int64_t H, int dt,
                                 void *out, void *stream) {
    if (w8a8_status s = moe_rows(T, top, H, H)) return s;
    if (!mx_dtype_ok(dt)) return W8A8_ERR_DTYPE;
    if (T == 0) return W8A8_OK;
    if (!rows || !slot_pos || !out || (weighted && !weights)) return W8A8_ERR_NULL;
    const int64_t size = dtype_size(dt);
    if (odd(rows, size) || odd(out, size) || odd(slot_pos, 4) || odd(weights, 4))
        return W8A8_ERR_ALIGN;
    return hip_status(moe::launch_combine(rows, slot_pos, weights, T, (int)top, (int)H, dt, out,
                                          static_cast<hipStream_t>(stream)));
}

w8a8_status moe_gather_backward(const void *d_rows, const int32_t *slot_pos, int64_t T,
                                int64_t top, int64_t H, mxfp4_dtype dtype, void *d_x,
                                void *stream) {
    return combine_entry(d_rows, slot_pos, nullptr, false, T, top, H, selector(&dtype), d_x, stream);
}

w8a8_status moe_combine(const void *rows, const int32_t *slot_pos, const float *weights,
                        int64_t T, int64_t top, int64_t H, mxfp4_dtype dtype, void *out,
                        void *stream) {
    return combine_entry(rows, slot_pos, weights, true, T, top, H, selector(&dtype), out, stream);
}

w8a8_status moe_combine_backward(const void *d_out, int64_t ldd, const void *rows,
                                 const int32_t *slot_pos, const float *weights, int64_t T,
                                 int64_t top, int64_t H, mxfp4_dtype dtype, void *d_rows,
                                 float *d_weights, void *stream) {
    if (w8a8_status s = moe_rows(T, top, H, ldd)) return s;
    const int dt = selector(&dtype);
    if (!mx_dtype_ok(dt)) return W8A8_ERR_DTYPE;
    if (T == 0) return W8A8_OK;
    if (!d_out || !rows || !slot_pos || !weights || !d_rows) return W8A8_ERR_NULL;
    const int64_t size = dtype_size(dt);
    if (odd(d_out, size) || odd(rows, size) || odd(d_rows, size) || odd(slot_pos, 4) ||
        odd(weights, 4) || odd(d_weights, 4))
        return W8A8_ERR_ALIGN;
    return hip_status(moe::launch_combine_backward(d_out, ldd, rows, slot_pos, weights, T, (int)top,
                                                   (int)H, dt, d_rows, d_weights,
                                                   static_cast<hipStream_t>(stream)));
}

// Checks shared by the experts' products, then the launch.
static w8a8_status expert_entry(const uint8_t *xq, const uint8_t *xs, int64_t T,
                                const int32_t *row_token, int64_t S, const int32_t *offsets,
                                int64_t E, const uint8_t *wq, const uint8_t *ws, int64_t N,
                                int64_t K, int epilogue, const mxfp4::Output &o, void *stream) {
    if (w8a8_status s = mx_shape(S, K)) return s;
    if (w8a8_status s = mx_shape(T, K)) return s;
    if (w8a8_status s = mx_weight(N, K)) return s;
    if (w8a8_status s = mx_out(S, N)) return s;
    if (E <= 0 || E > MOE_MAX_EXPERTS || (!row_token && T != S) || (S > 0 && T == 0))
        return W8A8_ERR_SHAPE;
    if (row_token)
        if (w8a8_status s = mx_tokens(T, K)) return s;
    if (S == 0) return W8A8_OK;
    if (!mxfp4::product_fits(mxfp4::Rows{S, E, true}, (int)N, (int)K, epilogue)) return W8A8_ERR_SHAPE;
    if (!xq || !xs || !offsets || !wq || !ws) return W8A8_ERR_NULL;
    if (epilogue == mxfp4::kSwiglu ? !o.codes || !o.scales : !o.out) return W8A8_ERR_NULL;
    if (misaligned(xq) || misaligned(xs) || misaligned(wq) || misaligned(ws) || misaligned(o.out) ||
        misaligned(o.codes) || misaligned(o.scales) || odd(offsets, 4) || odd(row_token, 4))
        return W8A8_ERR_ALIGN;
    const mxfp4::Groups g{offsets, row_token, (int)E, (int)S, (int)T};
    return hip_status(mxfp4::launch_gemm(xq, xs, wq, ws, g, (int)N, (int)K, epilogue, o,
                                         static_cast<hipStream_t>(stream)));
}

// Not part of the interface (the tests ask it which sizes reach which kernel): the form of a
// product's workgroups on a device of `cus` compute units, as stream * 10^9 + rows * 10^6 +
// channels * 10^3 + wavefronts.
extern "C" int mxfp4_debug_form(int64_t S, int64_t E, int grouped, int64_t N, int64_t K, int epilogue,
                                int64_t cus) {
    const mxfp4::Form f = mxfp4::product_form(mxfp4::Rows{S, E, grouped != 0}, (int)N, (int)K, epilogue, cus);
    return (f.stream ? 1000000000 : 0) + f.rows * 1000000 + f.channels * 1000 + f.waves;
}

w8a8_status mxfp4_expert_gemm(const uint8_t *xq, const uint8_t *xs, int64_t T,
                              const int32_t *row_token, int64_t S, const int32_t *offsets,
                              int64_t E, const uint8_t *wq, const uint8_t *ws, int64_t N,
                              int64_t K, mxfp4_dtype dtype, void *out, void *stream) {
    const int dt = selector(&dtype);
    if (!mx_dtype_ok(dt)) return W8A8_ERR_DTYPE;
    return expert_entry(xq, xs, T, row_token, S, offsets, E, wq, ws, N, K, dt,
                        mxfp4::Output{out, nullptr, nullptr}, stream);
}

w8a8_status mxfp4_expert_swiglu(const uint8_t *xq, const uint8_t *xs, int64_t T,
                                const int32_t *row_token, int64_t S, const int32_t *offsets,
                                int64_t E, const uint8_t *wq, const uint8_t *ws, int64_t F,
                                int64_t K, uint8_t *hq, uint8_t *hs, void *stream) {
    if (w8a8_status s = mx_shape(S, F)) return s;  // the hidden rows
    return expert_entry(xq, xs, T, row_token, S, offsets, E, wq, ws, 2 * F, K, mxfp4::kSwiglu,
                        mxfp4::Output{nullptr, hq, hs}, stream);
}

// Parts of mxfp4_moe's workspace, in bytes from its start.
struct MoeParts {
    int64_t offsets, slot_pos, row_token, sort, sort_bytes, xq, xs, hq, hs, y, total;
};

static w8a8_status moe_parts(int64_t T, int64_t top, int64_t E, int64_t H, int64_t F,
                             MoeParts &p) {
    if (w8a8_status s = moe_shape(T, top)) return s;
    if (E <= 0 || E > MOE_MAX_EXPERTS) return W8A8_ERR_SHAPE;
    const int64_t S = T * top;
    if (w8a8_status s = mx_shape(S, H)) return s;
    if (w8a8_status s = mx_shape(S, F)) return s;
    if (w8a8_status s = mx_weight(H, F)) return s;
    if (w8a8_status s = mx_weight(2 * F, H)) return s;
    if (w8a8_status s = mx_out(S, 2 * F)) return s;
    if (w8a8_status s = mx_out(S, H)) return s;
    if (w8a8_status s = mx_tokens(T, H)) return s;  // so the sort's grid holds the tokens' quantization too
    int64_t at = 0;
    auto take = [&](int64_t bytes) { const int64_t b = at; at += align256(bytes); return b; };
    p.offsets = take((E + 1) * 4);
    p.slot_pos = take(S * 4);
    p.row_token = take(S * 4);
    p.sort_bytes = moe_sort_workspace(S, E);
    p.sort = take(p.sort_bytes);
    p.xq = take(mx_codes(T, H));
    p.xs = take(mx_scales(T, H));
    p.hq = take(mx_codes(S, F));
    p.hs = take(mx_scales(S, F));
    p.y = take(S * H * 4);  // the experts' outputs stay in fp32 up to their weighted sum
    p.total = at;
    return W8A8_OK;
}

int64_t mxfp4_moe_workspace(int64_t T, int64_t top, int64_t E, int64_t H, int64_t F,
                            mxfp4_dtype dtype) {
    MoeParts p;
    const int dt = selector(&dtype);
    if (T <= 0 || !mx_dtype_ok(dt) || moe_parts(T, top, E, H, F, p) != W8A8_OK) return 0;
    return p.total;
}

w8a8_status mxfp4_moe(const void *x, int64_t ldx, mxfp4_dtype dtype, int64_t T, int64_t H,
                      const void *expert_ids, int ids_bits, const float *weights, int64_t top,
                      int64_t E, const uint8_t *w13q, const uint8_t *w13s, const uint8_t *w2q,
                      const uint8_t *w2s, int64_t F, void *out, void *workspace,
                      int64_t workspace_bytes, void *stream) {
    const int dt = selector(&dtype);
    if (!mx_dtype_ok(dt)) return W8A8_ERR_DTYPE;
    if (ids_bits != 32 && ids_bits != 64) return W8A8_ERR_DTYPE;
    MoeParts p;
    if (w8a8_status s = moe_parts(T, top, E, H, F, p)) return s;
    if (ldx < H || ldx > INT_MAX) return W8A8_ERR_SHAPE;
    if (T > 0 && workspace_bytes < p.total) return W8A8_ERR_SHAPE;
    if (T == 0) return W8A8_OK;
    if (!x || !expert_ids || !weights || !w13q || !w13s || !w2q || !w2s || !out || !workspace)
        return W8A8_ERR_NULL;
    if (misaligned(x) || misaligned(w13q) || misaligned(w13s) || misaligned(w2q) ||
        misaligned(w2s) || misaligned(out) || misaligned(workspace) || odd(weights, 4) ||
        odd(expert_ids, ids_bits / 8) || ldx * dtype_size(dt) % 16 != 0)
        return W8A8_ERR_ALIGN;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    int32_t *offsets = reinterpret_cast<int32_t *>(ws + p.offsets);
    int32_t *slot_pos = reinterpret_cast<int32_t *>(ws + p.slot_pos);
    int32_t *row_token = reinterpret_cast<int32_t *>(ws + p.row_token);
    const int64_t S = T * top;
    if (mxfp4::few_slots(S, H, F)) {
        const mxfp4::Ids slots{expert_ids, ids_bits, (int)top};
        hipStream_t st = static_cast<hipStream_t>(stream);
        if (w8a8_status s = hip_status(mxfp4::launch_moe_up(x, ldx, dt, slots, (int)S, (int)E, w13q, w13s, (int)F,
                                                            (int)H, ws + p.hq, ws + p.hs, st)))
            return s;
        return hip_status(mxfp4::launch_moe_down(ws + p.hq, ws + p.hs, slots, weights, (int)T, (int)E, w2q, w2s,
                                                 (int)H, (int)F, dt, out, st));
    }
    if (w8a8_status s = hip_status(moe::launch_sort_quantize(
            expert_ids, ids_bits == 64, S, (int)top, (int)E, offsets, slot_pos, row_token,
            ws + p.sort, x, ldx, T, (int)H, dt, ws + p.xq, ws + p.xs,
            static_cast<hipStream_t>(stream))))
        return s;
    if (w8a8_status s = mxfp4_expert_swiglu(ws + p.xq, ws + p.xs, T, row_token, S, offsets, E, w13q,
                                            w13s, F, H, ws + p.hq, ws + p.hs, stream))
        return s;
    if (w8a8_status s = mxfp4_expert_gemm(ws + p.hq, ws + p.hs, S, nullptr, S, offsets, E, w2q, w2s,
                                          H, F, MXFP4_F32, ws + p.y, stream))
        return s;
    return hip_status(moe::launch_combine_layer(reinterpret_cast<const float *>(ws + p.y), slot_pos, weights, T,
                                                (int)top, (int)H, dt, out, static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------- around a layer

static bool act_ok(int a) { return a >= W8A8_ACT_NONE && a <= W8A8_ACT_SILU; }

w8a8_status w8a8_gemm_act(const int8_t *xq, const float *x_scale, int64_t M, const int8_t *wq,
                          const float *w_scale, int64_t N, int64_t K, const float *bias,
                          w8a8_activation activation, const void *residual, int64_t ldr, void *out,
                          void *stream) {
    if (M < 0 || N <= 0 || N % 16 != 0 || too_big(M, N)) return W8A8_ERR_SHAPE;
    if (w8a8_status s = check_k(K)) return s;
    const int a = selector(&activation);
    if (!act_ok(a)) return W8A8_ERR_DTYPE;
    if ((M + 127) / 128 > INT_MAX / ((N + 127) / 128)) return W8A8_ERR_SHAPE;  // grid.x
    if (residual && (ldr < N || ldr > INT_MAX)) return W8A8_ERR_SHAPE;
    if (M == 0) return W8A8_OK;
    if (!dense_launch(M, N, K)) return W8A8_ERR_SHAPE;
    if (!xq || !x_scale || !wq || !w_scale || !out) return W8A8_ERR_NULL;
    if (misaligned(xq) || misaligned(x_scale) || misaligned(wq) || misaligned(w_scale) ||
        misaligned(out) || misaligned(bias) || misaligned(residual) || (residual && ldr % 8 != 0))
        return W8A8_ERR_ALIGN;
    const w8a8::ActEpilogue ep{bias, residual, ldr, a};
    return hip_status(w8a8::launch_gemm_act(xq, x_scale, (int)M, wq, w_scale, (int)N, (int)K, out, ep,
                                            static_cast<hipStream_t>(stream)));
}

// Not part of the interface (the tests ask it which sizes reach which kernel).
int w8a8_act_debug_form(int64_t M, int64_t N, int64_t K) { return w8a8::act_form(M, N, K); }

static w8a8_status linear16_shape(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || M >= (1 << 27) || N <= 0 || K <= 0 || N % 8 != 0 || K % 8 != 0 ||
        N > W16A16_MAX_WIDTH || K > W16A16_MAX_WIDTH)
        return W8A8_ERR_SHAPE;
    const int64_t most = (int64_t)1 << 35;  // tiles are counted in 32 bits
    if (M * N > most || M * K > most || N * K > most) return W8A8_ERR_SHAPE;
    return W8A8_OK;
}

// Not part of the interface (the tests ask them which sizes reach which kernel): of a product of a 16-bit
// layer (0 forward, 1 d_x, 2 d_w, 3 and 4 those in one launch), 10^6 for the kernel of few rows,
// otherwise the tiles' form * 10^5 + (whole tiles) * 10^4 + workgroups of the others.
int w16a16_debug_form(int64_t M, int64_t N, int64_t K, int product) {
    if (product == 0) {
        const linear16::ForwardPlan p = linear16::plan_forward(M, N, K);
        return p.rows ? 1000000 : p.tiles.form * 100000 + (p.tiles.whole > 0) * 10000 + p.tiles.splits;
    }
    const linear16::BackwardPlan p = linear16::plan_backward(M, N, K);
    const linear16::Plan &t = product == 1 ? p.x : product == 2 ? p.w : product == 3 ? p.both.x : p.both.w;
    return t.form * 100000 + (t.whole > 0) * 10000 + t.splits;
}

int64_t w16a16_linear_workspace(int64_t M, int64_t N, int64_t K) {
    return linear16_shape(M, N, K) == W8A8_OK ? linear16::plan_forward(M, N, K).workspace() : 0;
}

w8a8_status w16a16_linear(const void *x, int64_t ldx, int64_t M, const void *w, int64_t N,
                          int64_t K, w4a16_dtype dtype, const float *bias,
                          w8a8_activation activation, const void *residual, int64_t ldr, void *pre,
                          void *out, void *workspace, int64_t workspace_bytes, void *stream) {
    if (w8a8_status s = linear16_shape(M, N, K)) return s;
    const int dt = selector(&dtype), a = selector(&activation);
    if ((dt != W4A16_BF16 && dt != W4A16_F16) || !act_ok(a)) return W8A8_ERR_DTYPE;
    linear16::ForwardPlan plan = linear16::plan_forward(M, N, K);
    if (M <= linear16::kNoWorkspaceRows && workspace_bytes >= 0 && workspace_bytes < plan.workspace()) plan.rows = true;
    const int64_t need = plan.workspace();
    if (ldx < K || ldx > INT_MAX || (residual && (ldr < N || ldr > INT_MAX)) || workspace_bytes < need)
        return W8A8_ERR_SHAPE;
    if (M == 0) return W8A8_OK;
    if (!x || !w || !out || (need && !workspace)) return W8A8_ERR_NULL;
    if (misaligned(x) || misaligned(w) || misaligned(out) || misaligned(bias) || misaligned(residual) ||
        misaligned(pre) || misaligned(workspace) || ldx % 8 != 0 || (residual && ldr % 8 != 0))
        return W8A8_ERR_ALIGN;
    const linear16::Epilogue ep{bias, residual, ldr, pre, out, a};
    return hip_status(linear16::launch_forward(plan, x, ldx, M, w, N, K, dt == W4A16_F16, ep, workspace,
                                               static_cast<hipStream_t>(stream)));
}

int64_t w16a16_linear_backward_workspace(int64_t M, int64_t N, int64_t K) {
    return linear16_shape(M, N, K) == W8A8_OK ? linear16::plan_backward(M, N, K).workspace : 0;
}

w8a8_status w16a16_linear_backward(const void *d_out, int64_t ldd, const void *x, int64_t ldx,
                                   const void *w, const void *pre, int64_t M, int64_t N, int64_t K,
                                   w4a16_dtype dtype, w8a8_activation activation, void *d_pre,
                                   void *d_x, void *d_w, float *d_bias, void *workspace,
                                   int64_t workspace_bytes, void *stream) {
    if (w8a8_status s = linear16_shape(M, N, K)) return s;
    const int dt = selector(&dtype), a = selector(&activation);
    if ((dt != W4A16_BF16 && dt != W4A16_F16) || !act_ok(a)) return W8A8_ERR_DTYPE;
    const linear16::BackwardPlan plan = linear16::plan_backward(M, N, K);
    const int64_t need = plan.workspace;
    if (ldd < N || ldd > INT_MAX || ldx < K || ldx > INT_MAX || workspace_bytes < need)
        return W8A8_ERR_SHAPE;
    const bool slope = a != W8A8_ACT_NONE;
    if (M > 0 && (!d_out || (d_w && !x) || (d_x && !w) || (slope && (!pre || !d_pre)) || (need && !workspace)))
        return W8A8_ERR_NULL;
    if (misaligned(d_out) || misaligned(x) || misaligned(w) || misaligned(pre) || misaligned(d_pre) ||
        misaligned(d_x) || misaligned(d_w) || misaligned(d_bias) || misaligned(workspace) ||
        ldd % 8 != 0 || ldx % 8 != 0)
        return W8A8_ERR_ALIGN;
    return hip_status(linear16::launch_backward(plan, d_out, ldd, x, ldx, w, pre, M, N, K, dt == W4A16_F16, a,
                                                d_pre, d_x, d_w, d_bias, workspace,
                                                static_cast<hipStream_t>(stream)));
}

// Sizes, type and scalars of a block norm.
static w8a8_status norm_shape(int64_t T, int64_t H) {
    // above 512 rows, a row of up to 512 elements has at most 64 threads and a longer one (128 to 1024 by type and
    // width) fewer than H / 4: less than 2^30 and 2^32 threads in all
    if (T < 0 || T >= (1 << 24) || H <= 0 || H > BLOCK_NORM_MAX_H || T * H > ((int64_t)1 << 34))
        return W8A8_ERR_SHAPE;
    return W8A8_OK;
}

static w8a8_status norm_scalars(float scale, float eps) {
    return std::isfinite(scale) && std::isfinite(eps) && eps > 0 ? W8A8_OK : W8A8_ERR_VALUE;
}

static bool short_rows(const void *rows, int64_t ld, int64_t H) {
    return rows && (ld < H || ld > INT_MAX);
}

static bool bad_gate(const void *gate, int64_t ldg, int64_t size) {
    return gate && (ldg == 0 ? misaligned(gate) : odd(gate, size));
}

static w8a8_status norm_entry(block::Forward a, int dt, int out, void *stream) {
    if (w8a8_status s = norm_shape(a.T, a.H)) return s;
    if (!mx_dtype_ok(dt)) return W8A8_ERR_DTYPE;
    if (w8a8_status s = norm_scalars(a.scale, a.eps)) return s;
    if (a.ldr < a.H || a.ldr > INT_MAX || short_rows(a.y, a.ldy, a.H) ||
        (a.y && a.ldg != 0 && short_rows(a.gate, a.ldg, a.H)))
        return W8A8_ERR_SHAPE;
    if (out != block::kSame && a.H % (out == block::kInt8 ? 16 : 32) != 0) return W8A8_ERR_SHAPE;
    if (a.T == 0) return W8A8_OK;
    if (!a.residual || (a.y && !a.new_residual) || !a.out || (out != block::kSame && !a.out_scale))
        return W8A8_ERR_NULL;
    const int64_t size = dtype_size(dt);
    if (odd(a.residual, size) || odd(a.y, size) || odd(a.new_residual, size) ||
        (a.y && bad_gate(a.gate, a.ldg, size)) || misaligned(a.weight) || misaligned(a.post_weight) ||
        (out == block::kSame ? odd(a.out, size) : misaligned(a.out) || misaligned(a.out_scale)))
        return W8A8_ERR_ALIGN;
    if (!a.y) a.gate = nullptr, a.post = 0;
    return hip_status(block::launch_forward(a, dt, out, static_cast<hipStream_t>(stream)));
}

static int clamp_h(int64_t H) { return H < 0 || H > INT_MAX ? 0 : (int)H; }  // 0 is refused

w8a8_status block_norm(const void *residual, int64_t ldr, const void *y, int64_t ldy,
                       int post_norm, const float *post_weight, const void *gate, int64_t ldg,
                       float scale, const float *weight, float eps, int64_t T, int64_t H,
                       mxfp4_dtype dtype, void *new_residual, void *out, void *stream) {
    return norm_entry({residual, y, gate, ldr, ldy, ldg, post_weight, weight, post_norm, scale, eps, T,
                       clamp_h(H), new_residual, out, nullptr},
                      selector(&dtype), block::kSame, stream);
}

w8a8_status block_norm_w8a8(const void *residual, int64_t ldr, const void *y, int64_t ldy,
                            int post_norm, const float *post_weight, const void *gate,
                            int64_t ldg, float scale, const float *weight, float eps, int64_t T,
                            int64_t H, mxfp4_dtype dtype, void *new_residual, int8_t *xq,
                            float *x_scale, void *stream) {
    return norm_entry({residual, y, gate, ldr, ldy, ldg, post_weight, weight, post_norm, scale, eps, T,
                       clamp_h(H), new_residual, xq, x_scale},
                      selector(&dtype), block::kInt8, stream);
}

w8a8_status block_norm_mxfp4(const void *residual, int64_t ldr, const void *y, int64_t ldy,
                             int post_norm, const float *post_weight, const void *gate,
                             int64_t ldg, float scale, const float *weight, float eps, int64_t T,
                             int64_t H, mxfp4_dtype dtype, void *new_residual, uint8_t *codes,
                             uint8_t *scales, void *stream) {
    return norm_entry({residual, y, gate, ldr, ldy, ldg, post_weight, weight, post_norm, scale, eps, T,
                       clamp_h(H), new_residual, codes, scales},
                      selector(&dtype), block::kMxfp4, stream);
}

int64_t block_norm_backward_workspace(int64_t T, int64_t H) {
    return norm_shape(T, H) == W8A8_OK ? block::backward_workspace(T, H) : 0;
}

w8a8_status block_norm_backward(const void *d_out, int64_t ldo, const void *d_new, int64_t ldn,
                                const void *new_residual, int64_t ldr, const void *y, int64_t ldy,
                                int post_norm, const float *post_weight, const void *gate,
                                int64_t ldg, float scale, const float *weight, float eps,
                                int64_t T, int64_t H, mxfp4_dtype dtype, void *d_residual,
                                void *d_y, void *d_gate, float *d_weight, float *d_post_weight,
                                void *workspace, int64_t workspace_bytes, void *stream) {
    if (w8a8_status s = norm_shape(T, H)) return s;
    const int dt = selector(&dtype);
    if (!mx_dtype_ok(dt)) return W8A8_ERR_DTYPE;
    if (w8a8_status s = norm_scalars(scale, eps)) return s;
    if (!y && T > 0) gate = nullptr, post_norm = 0;
    if (!gate) d_gate = nullptr;
    if (!post_norm) d_post_weight = nullptr;
    const int64_t need = block::backward_workspace(T, H);
    if (ldo < H || ldo > INT_MAX || ldr < H || ldr > INT_MAX || short_rows(d_new, ldn, H) ||
        short_rows(y, ldy, H) || (ldg != 0 && short_rows(gate, ldg, H)) || workspace_bytes < need)
        return W8A8_ERR_SHAPE;
    if (T > 0 && (!d_out || !new_residual || !d_residual || (y && !d_y) || !workspace))
        return W8A8_ERR_NULL;
    const int64_t size = dtype_size(dt);
    if (odd(d_out, size) || odd(d_new, size) || odd(new_residual, size) || odd(y, size) ||
        odd(d_residual, size) || odd(d_y, size) || bad_gate(gate, ldg, size) ||
        bad_gate(d_gate, ldg, size) || misaligned(weight) || misaligned(post_weight) ||
        misaligned(d_weight) || misaligned(d_post_weight) || misaligned(workspace))
        return W8A8_ERR_ALIGN;
    const block::Backward a{d_out, d_new, new_residual, y, gate, ldo, ldn, ldr, ldy, ldg, post_weight,
                            weight, post_norm, scale, eps, T, (int)H, d_residual, d_y, d_gate, d_weight,
                            d_post_weight, static_cast<float *>(workspace)};
    return hip_status(block::launch_backward(a, dt, static_cast<hipStream_t>(stream)));
}

const char *w8a8_status_string(int status) {
    switch (status) {
        case W8A8_OK: return "ok";
        case W8A8_ERR_NULL: return "a required pointer is NULL";
        case W8A8_ERR_SHAPE: return "a size is out of range or not a required multiple";
        case W8A8_ERR_ALIGN: return "a base pointer is not 16-byte aligned";
        case W8A8_ERR_K_OVERFLOW: return "K exceeds the int32-safe bound (128*128*K < 2^31)";
        case W8A8_ERR_BLOCKSIZE: return "BSR block size must be 64";
        case W8A8_ERR_DTYPE: return "unknown output dtype";
        case W8A8_ERR_HIP: return "HIP launch error (see w8a8_last_hip_error)";
        case W8A8_ERR_VALUE: return "a scalar is not finite or out of range";
        default: return "unknown status";
    }
}

int w8a8_last_hip_error(void) { return g_last_hip_error; }

}  // extern "C"
