// Internal kernel launchers behind the C ABI (w8a8_abi.cpp). Arguments are
// already validated when these run; each returns the HIP error of its launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w8a8 {

hipError_t launch_quantize_rows_bf16(const uint16_t *x, int64_t M, int K, int8_t *xq, float *xs,
                                     hipStream_t stream);
hipError_t launch_quantize_rows_f32(const float *x, int64_t M, int K, int8_t *xq, float *xs,
                                    hipStream_t stream);

struct Addmm;

// Dense GEMM: picks the weight-streaming kernel for M <= 64, the LDS-tiled
// MFMA kernel otherwise. With am non-null (bf16 output only) the epilogue is
// alpha * (acc * sa * sb) + beta * bias.
hipError_t launch_gemm(const int8_t *xq, const float *xs, int M, const int8_t *wq, const float *ws,
                       int N, int K, void *out, bool out_i32, hipStream_t stream,
                       const Addmm *am = nullptr);

// Epilogue act(acc * sa * sb + bias[n]) + residual[m, n] (bias and residual may be null; act an
// act::Activation), and the product with it: on the same kernels, or on tiles of its own.
struct ActEpilogue {
    const float *bias;
    const void *residual;  // bf16 rows, row stride ldr
    int64_t ldr;
    int act;
};
enum ActForm { kActStreaming, kActOwnStages, kAct64x64, kActTiles };
ActForm act_form(int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm_act(const int8_t *xq, const float *xs, int M, const int8_t *wq, const float *ws,
                           int N, int K, void *out, const ActEpilogue &ep, hipStream_t stream);

// Single-launch linear for M <= 64: quantize_rows of bf16 X fused into the
// weight-streaming GEMM, epilogue as launch_gemm's with am.
hipError_t launch_linear_decode(const uint16_t *x, int M, const int8_t *wq, const float *ws, int N,
                                int K, void *out, hipStream_t stream, const Addmm &am);

// 2:4 weights: compression of an int8 [N,K] weight (K % 64 == 0) into values
// [N,K/2] and meta [N,K/32], and the GEMM on the compressed weight.
hipError_t launch_compress24(const int8_t *wq, int N, int K, int8_t *values, uint32_t *meta,
                             hipStream_t stream);
hipError_t launch_sparse24_gemm(const int8_t *xq, const float *xs, int M, const int8_t *values,
                                const uint32_t *meta, const float *ws, int N, int K, void *out,
                                bool out_i32, hipStream_t stream);

// A launch holds fewer than 2^32 threads.
inline bool grid_fits(int64_t workgroups, int threads) { return workgroups * threads < ((int64_t)1 << 32); }

// Compute units of the current device (queried once per device).
int device_cu_count();

// Block-sparse GEMM; am (bf16 output only) selects the addmm epilogue.
hipError_t launch_bsr_gemm(const int8_t *xq, const float *xs, int M, int K, const int32_t *crow,
                           const int32_t *col, const int8_t *values, int nnzb, const float *ws,
                           int N, void *out, bool out_i32, hipStream_t stream,
                           const Addmm *am = nullptr);

}  // namespace w8a8

namespace w4a16 {

// W4A16 (16-bit values as uint16_t bit patterns: bf16, or binary16 when f16):
// standalone dequantization of packed 4-bit weights [N,K/2] (u4, or s4 when
// s4) with scales/zeros [N,K/G] into w [N,K], and the fused dequant GEMM
// out [M,N] = round(x [M,K] . w^T).
hipError_t launch_dequant(const uint8_t *wq4, const uint16_t *scales, const uint16_t *zeros, int N,
                          int K, int G, bool s4, bool f16, uint16_t *w, hipStream_t stream);
hipError_t launch_gemm(const uint16_t *x, int M, const uint8_t *wq4, const uint16_t *scales,
                       const uint16_t *zeros, int N, int K, int G, bool s4, bool f16,
                       uint16_t *out, hipStream_t stream);

}  // namespace w4a16

namespace mxfp4 {

struct Groups;
struct Output;
struct Ids;

// MXFP4 rows (dtype 0 bf16, 1 binary16, 2 binary32): x [M,K] with row stride
// ldx -> codes [M,K/2], scales [ceil(K/256),M,8], and back to out [M,K].
hipError_t launch_quantize(const void *x, int64_t ldx, int64_t M, int K, int dtype, uint8_t *codes,
                           uint8_t *scales, hipStream_t stream);
hipError_t launch_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t M, int K,
                             int dtype, void *out, hipStream_t stream);

// Product of MXFP4 rows and weights [E][N,K] (one weight without offsets);
// epilogue: a dtype, or 3 for SwiGLU + MXFP4.
hipError_t launch_gemm(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws,
                       const Groups &g, int N, int K, int epilogue, const Output &o,
                       hipStream_t stream);

// The single-launch layer for a few rows: x is quantized inside the
// weight-streaming product, by every workgroup for itself. Taken for up to 4
// rows and 8192 channels. A call then costs the host one launch instead of two
// (8.3 against 12.6 us) and the GPU no more: 4096 x 4096, M = 1 5.8 us against 6.0
// in two launches, M = 4 6.1 / 6.2, but M = 8 7.7 / 6.3; M = 1 with 16384 channels
// 18.5 / 11.1.
inline bool single_launch_linear(int64_t M, int64_t N) { return M <= 4 && N <= 8192; }
hipError_t launch_linear_decode(const void *x, int64_t ldx, int x_dtype, int M, const uint8_t *wq,
                                const uint8_t *ws, int N, int K, int out_dtype, void *out,
                                hipStream_t stream);

// The expert layer of a few slots, in two launches without a sort: the gate and
// up products with SwiGLU of every slot (x quantized inside) into hidden rows in
// slot order, and the down products with the weighted sum. Two slots of one
// expert read its weights twice, so it is for few slots, or small experts.
// Against the sort and four launches, us (4096 / 2048, bf16): 4 slots on 32 experts
// 18.2 / 22.2, 8 25.7 / 29.3, 16 41.8 / 37.9; 8 slots on 8 experts 23.7 / 25.8;
// experts of 1024 / 512: 4 slots 7.9 / 15.8, 16 8.7 / 16.7; 64 slots of 512 / 512
// 13.5 / 18.6.
inline bool few_slots(int64_t S, int64_t H, int64_t F) {
    return S <= 8 || (S <= 64 && S * H * F <= (1 << 24));
}
hipError_t launch_moe_up(const void *x, int64_t ldx, int dtype, const Ids &slots, int S, int E,
                         const uint8_t *wq, const uint8_t *ws, int F, int K, uint8_t *hq, uint8_t *hs,
                         hipStream_t stream);
hipError_t launch_moe_down(const uint8_t *hq, const uint8_t *hs, const Ids &slots, const float *weights,
                           int T, int E, const uint8_t *wq, const uint8_t *ws, int N, int K, int dtype,
                           void *out, hipStream_t stream);

}  // namespace mxfp4

namespace moe {

// Bytes of scratch that launch_sort needs for S slots.
int64_t sort_workspace(int64_t S, int64_t E);
hipError_t launch_sort(const void *ids, bool ids64, int64_t S, int top, int E, int32_t *offsets,
                       int32_t *slot_pos, int32_t *row_token, void *workspace, hipStream_t stream);
// The sort with the quantization of the T tokens x [T,H] in the same launch.
hipError_t launch_sort_quantize(const void *ids, bool ids64, int64_t S, int top, int E,
                                int32_t *offsets, int32_t *slot_pos, int32_t *row_token,
                                void *workspace, const void *x, int64_t ldx, int64_t T, int H,
                                int dtype, uint8_t *codes, uint8_t *scales, hipStream_t stream);
hipError_t launch_gather(const void *x, int64_t ldx, const int32_t *slot_pos, int64_t T, int top,
                         int H, int dtype, void *rows, hipStream_t stream);
// weights null: the plain sum (the gather's gradient)
hipError_t launch_combine(const void *rows, const int32_t *slot_pos, const float *weights,
                          int64_t T, int top, int H, int dtype, void *out, hipStream_t stream);
// the layer's sum: fp32 rows (16-byte aligned, H a multiple of 32) to out of dtype
hipError_t launch_combine_layer(const float *rows, const int32_t *slot_pos, const float *weights,
                                int64_t T, int top, int H, int dtype, void *out, hipStream_t stream);
hipError_t launch_combine_backward(const void *d_out, int64_t ldd, const void *rows,
                                   const int32_t *slot_pos, const float *weights, int64_t T,
                                   int top, int H, int dtype, void *d_rows, float *d_weights,
                                   hipStream_t stream);

}  // namespace moe

namespace block {

struct Forward;
struct Backward;

// The block norm (norm.hpp's arguments; dtype 0 bf16, 1 binary16, 2 binary32;
// out 0 rows of dtype, 1 int8 rows, 2 MXFP4 rows) and its gradients.
hipError_t launch_forward(const Forward &a, int dtype, int out, hipStream_t stream);

// Bytes for the partial sums that the backward pass's workgroups leave.
int64_t backward_workspace(int64_t T, int64_t H);
hipError_t launch_backward(const Backward &a, int dtype, hipStream_t stream);

}  // namespace block

namespace linear16 {

struct Epilogue;
struct ForwardPlan;
struct BackwardPlan;

// 16-bit products (bf16, or binary16 when f16): x [M,K] with row stride ldx times w [N,K] with
// the epilogue, and the gradients (null outputs are left out), by the plans of linear16.hpp for their
// sizes. d_pre is not written without an activation (it is d_out then).
hipError_t launch_forward(const ForwardPlan &plan, const void *x, int64_t ldx, int64_t M, const void *w, int64_t N, int64_t K,
                          bool f16, const Epilogue &ep, void *workspace, hipStream_t stream);
hipError_t launch_backward(const BackwardPlan &plan, const void *d_out, int64_t ldd, const void *x, int64_t ldx, const void *w,
                           const void *pre, int64_t M, int64_t N, int64_t K, bool f16, int act, void *d_pre,
                           void *d_x, void *d_w, float *d_bias, void *workspace, hipStream_t stream);

}  // namespace linear16
