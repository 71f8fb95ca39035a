"""Python binding of libw8a8.so (C ABI in include/w8a8.h): marshalling only.

Each function checks tensor dtypes, shapes and devices, allocates missing
outputs with torch.empty on the input's device, and passes raw device
pointers plus the current HIP stream, or `stream`, to the library function of
the same name. With `stream`, what the binding allocates (outputs and
workspaces) belongs to that stream, as if the call were made under
torch.cuda.stream(stream); the caller orders the rest: `stream` has to wait for
inputs and buffers of the caller's that other streams still write or read, other
streams for the outputs, and a tensor that is dropped while another stream than
its own uses it needs torch's record_stream. All arithmetic runs in the library's
kernels; there is no fallback. If libw8a8.so is absent, every entry point raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libw8a8.so")

W8A8_OK = 0
W8A8_ERR_NULL = -1
W8A8_ERR_SHAPE = -2
W8A8_ERR_ALIGN = -3
W8A8_ERR_K_OVERFLOW = -4
W8A8_ERR_BLOCKSIZE = -5
W8A8_ERR_DTYPE = -6
W8A8_ERR_HIP = -7
W8A8_ERR_VALUE = -8
W8A8_OUT_BF16 = 0
W8A8_OUT_I32 = 1
W8A8_MAX_K = 131056
W8A8_FUSED_MAX_M = 64

_lib = None


class W8A8Error(RuntimeError):
    def __init__(self, status: int, fn: str):
        lib = load()
        msg = lib.w8a8_status_string(status).decode()
        if status == W8A8_ERR_HIP:
            msg += f" (hipError_t {lib.w8a8_last_hip_error()})"
        super().__init__(f"{fn}: status {status}: {msg}")
        self.status = status


def load():
    """Load libw8a8.so and declare its C signatures (raises if not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built: run __graft_entry__.build() first")
    lib = ctypes.CDLL(LIB_PATH)
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.w8a8_quantize_rows.argtypes = [p, i64, i64, p, p, p]
    lib.w8a8_quantize_rows_f32.argtypes = [p, i64, i64, p, p, p]
    lib.w8a8_gemm.argtypes = [p, p, i64, p, p, i64, i64, p, i32, p]
    lib.w8a8_bsr_gemm.argtypes = [p, p, i64, i64, p, p, p, i64, i64, p, i64, p, i32, p]
    f32 = ctypes.c_float
    lib.w8a8_gemm_addmm.argtypes = [p, p, i64, p, p, i64, i64, p, f32, f32, p, p]
    lib.w8a8_bsr_gemm_addmm.argtypes = [p, p, i64, i64, p, p, p, i64, i64, p, i64, p, f32, f32,
                                        p, p]
    lib.w8a8_fused_linear.argtypes = [p, i64, i64, p, p, i64, p, f32, f32, p, p]
    lib.w8a8_compress24.argtypes = [p, i64, i64, p, p, p]
    lib.w8a8_sparse24_gemm.argtypes = [p, p, i64, p, p, p, i64, i64, p, i32, p]
    lib.w4a16_dequant.argtypes = [p, p, p, i64, i64, i64, i32, i32, p, p]
    lib.w4a16_gemm.argtypes = [p, i64, p, p, p, i64, i64, i64, i32, i32, p, p]
    for fn in ("w8a8_quantize_rows", "w8a8_quantize_rows_f32", "w8a8_gemm", "w8a8_gemm_addmm",
               "w8a8_fused_linear", "w8a8_bsr_gemm", "w8a8_bsr_gemm_addmm", "w8a8_compress24",
               "w8a8_sparse24_gemm",
               "w4a16_dequant", "w4a16_gemm"):
        getattr(lib, fn).restype = i32
    lib.mxfp4_quantize_rows.argtypes = [p, i64, i64, i64, i32, p, p, p]
    lib.mxfp4_dequantize_rows.argtypes = [p, p, i64, i64, i32, p, p]
    lib.mxfp4_gemm.argtypes = [p, p, i64, p, p, i64, i64, i32, p, p]
    lib.mxfp4_linear.argtypes = [p, i64, i32, i64, p, p, i64, i64, i32, p, p, i64, p]
    lib.mxfp4_expert_gemm.argtypes = [p, p, i64, p, i64, p, i64, p, p, i64, i64, i32, p, p]
    lib.mxfp4_expert_swiglu.argtypes = [p, p, i64, p, i64, p, i64, p, p, i64, i64, p, p, p]
    lib.mxfp4_moe.argtypes = [p, i64, i32, i64, i64, p, i32, p, i64, i64, p, p, p, p, i64, p, p,
                              i64, p]
    lib.moe_sort.argtypes = [p, i32, i64, i64, i64, p, p, p, p, i64, p]
    lib.moe_gather.argtypes = [p, i64, p, i64, i64, i64, i32, p, p]
    lib.moe_gather_backward.argtypes = [p, p, i64, i64, i64, i32, p, p]
    lib.moe_combine.argtypes = [p, p, p, i64, i64, i64, i32, p, p]
    lib.moe_combine_backward.argtypes = [p, i64, p, p, p, i64, i64, i64, i32, p, p, p]
    for fn in ("mxfp4_quantize_rows", "mxfp4_dequantize_rows", "mxfp4_gemm", "mxfp4_linear",
               "mxfp4_expert_gemm", "mxfp4_expert_swiglu", "mxfp4_moe", "moe_sort", "moe_gather",
               "moe_gather_backward", "moe_combine", "moe_combine_backward"):
        getattr(lib, fn).restype = i32
    lib.mxfp4_linear_workspace.argtypes = [i64, i64, i64]
    lib.moe_sort_workspace.argtypes = [i64, i64]
    lib.mxfp4_moe_workspace.argtypes = [i64, i64, i64, i64, i64, i32]
    for fn in ("mxfp4_linear_workspace", "moe_sort_workspace", "mxfp4_moe_workspace"):
        getattr(lib, fn).restype = i64
    lib.w8a8_gemm_act.argtypes = [p, p, i64, p, p, i64, i64, p, i32, p, i64, p, p]
    lib.w16a16_linear.argtypes = [p, i64, i64, p, i64, i64, i32, p, i32, p, i64, p, p, p, i64, p]
    lib.w16a16_linear_backward.argtypes = [p, i64, p, i64, p, p, i64, i64, i64, i32, i32, p, p, p, p,
                                           p, i64, p]
    norm = [p, i64, p, i64, i32, p, p, i64, f32, p, f32, i64, i64, i32, p]
    lib.block_norm.argtypes = norm + [p, p]
    lib.block_norm_w8a8.argtypes = lib.block_norm_mxfp4.argtypes = norm + [p, p, p]
    lib.block_norm_backward.argtypes = [p, i64, p, i64, p, i64, p, i64, i32, p, p, i64, f32, p, f32,
                                        i64, i64, i32, p, p, p, p, p, p, i64, p]
    for fn in ("w8a8_gemm_act", "w16a16_linear", "w16a16_linear_backward", "block_norm",
               "block_norm_w8a8", "block_norm_mxfp4", "block_norm_backward"):
        getattr(lib, fn).restype = i32
    lib.w16a16_linear_workspace.argtypes = [i64, i64, i64]
    lib.w16a16_linear_backward_workspace.argtypes = [i64, i64, i64]
    lib.block_norm_backward_workspace.argtypes = [i64, i64]
    for fn in ("w16a16_linear_workspace", "w16a16_linear_backward_workspace",
               "block_norm_backward_workspace"):
        getattr(lib, fn).restype = i64
    lib.w8a8_status_string.argtypes = [i32]
    lib.w8a8_status_string.restype = ctypes.c_char_p
    lib.w8a8_last_hip_error.argtypes = []
    lib.w8a8_last_hip_error.restype = i32
    _lib = lib
    return lib


def _new(shape, dtype, like, stream):
    """A new tensor on `like`'s device in the pool of the stream that will write it: the allocator
    hands out memory that was freed with work still queued on its stream."""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=like.device)  # the quickest form
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=dtype, device=like.device)


def _stream_handle(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _check_tensor(t: torch.Tensor, name: str, dtype, ndim: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _default_beta(bias, beta):
    """beta of an addmm call: as given, else 1 with a bias and 0 without (the C ABI
    rejects a nonzero beta without a bias)."""
    if beta is None:
        return 1.0 if bias is not None else 0.0
    return beta


def _call(fn: str, *args):
    st = getattr(load(), fn)(*args)
    if st != W8A8_OK:
        raise W8A8Error(st, fn)


def _quantize(fn, x, xq, x_scale, stream, dtype):
    _check_tensor(x, "x", dtype, 2)
    M, K = x.shape
    if xq is None:
        xq = _new((M, K), torch.int8, x, stream)
    if x_scale is None:
        x_scale = _new((M,), torch.float32, x, stream)
    _check_tensor(xq, "xq", torch.int8, 2)
    _check_tensor(x_scale, "x_scale", torch.float32, 1)
    if tuple(xq.shape) != (M, K) or tuple(x_scale.shape) != (M,):
        raise ValueError("output shapes")
    _call(fn, x.data_ptr(), M, K, xq.data_ptr(), x_scale.data_ptr(), _stream_handle(stream))
    return xq, x_scale


def w8a8_quantize_rows(x, xq=None, x_scale=None, stream=None):
    """bf16 [M,K] -> (int8 [M,K], fp32 [M]) per-row absmax/127 quantization."""
    return _quantize("w8a8_quantize_rows", x, xq, x_scale, stream, torch.bfloat16)


def w8a8_quantize_rows_f32(x, xq=None, x_scale=None, stream=None):
    """fp32 [M,K] -> (int8 [M,K], fp32 [M]); per-output-channel weight preparation."""
    return _quantize("w8a8_quantize_rows_f32", x, xq, x_scale, stream, torch.float32)


def _out(out, M, N, out_dtype, like, stream):
    tdtype = torch.bfloat16 if out_dtype == W8A8_OUT_BF16 else torch.int32
    if out is None:
        out = _new((M, N), tdtype, like, stream)
    _check_tensor(out, "out", tdtype, 2)
    if tuple(out.shape) != (M, N):
        raise ValueError("out shape")
    return out


def _out_dtype(out_dtype) -> int:
    if out_dtype in ("bf16", torch.bfloat16, W8A8_OUT_BF16):
        return W8A8_OUT_BF16
    if out_dtype in ("i32", torch.int32, W8A8_OUT_I32):
        return W8A8_OUT_I32
    raise ValueError(f"out_dtype {out_dtype!r}")


def w8a8_gemm(xq, x_scale, wq, w_scale, out=None, out_dtype="bf16", stream=None):
    """out [M,N] = bf16(sum_k xq[m,k] wq[n,k] * x_scale[m] * w_scale[n]) (or int32 acc)."""
    od = _out_dtype(out_dtype)
    _check_tensor(xq, "xq", torch.int8, 2)
    _check_tensor(x_scale, "x_scale", torch.float32, 1)
    _check_tensor(wq, "wq", torch.int8, 2)
    _check_tensor(w_scale, "w_scale", torch.float32, 1)
    M, K = xq.shape
    N, K2 = wq.shape
    if K2 != K or tuple(x_scale.shape) != (M,) or tuple(w_scale.shape) != (N,):
        raise ValueError("operand shapes")
    out = _out(out, M, N, od, xq, stream)
    _call("w8a8_gemm", xq.data_ptr(), x_scale.data_ptr(), M, wq.data_ptr(), w_scale.data_ptr(),
          N, K, out.data_ptr(), od, _stream_handle(stream))
    return out


def w8a8_gemm_addmm(xq, x_scale, wq, w_scale, bias=None, alpha=1.0, beta=None, out=None,
                    stream=None):
    """out [M,N] = bf16(alpha * (sum_k xq[m,k] wq[n,k] * x_scale[m] * w_scale[n]) + beta * bias[n]);
    bias None means no bias term; beta defaults to 1 with a bias and 0 without."""
    beta = _default_beta(bias, beta)
    _check_tensor(xq, "xq", torch.int8, 2)
    _check_tensor(x_scale, "x_scale", torch.float32, 1)
    _check_tensor(wq, "wq", torch.int8, 2)
    _check_tensor(w_scale, "w_scale", torch.float32, 1)
    M, K = xq.shape
    N, K2 = wq.shape
    if K2 != K or tuple(x_scale.shape) != (M,) or tuple(w_scale.shape) != (N,):
        raise ValueError("operand shapes")
    if bias is not None:
        _check_tensor(bias, "bias", torch.float32, 1)
        if tuple(bias.shape) != (N,):
            raise ValueError("bias shape")
    out = _out(out, M, N, _out_dtype("bf16"), xq, stream)
    _call("w8a8_gemm_addmm", xq.data_ptr(), x_scale.data_ptr(), M, wq.data_ptr(),
          w_scale.data_ptr(), N, K, None if bias is None else bias.data_ptr(), float(alpha),
          float(beta), out.data_ptr(), _stream_handle(stream))
    return out


def w8a8_compress24(wq, values=None, meta=None, stream=None):
    """int8 [N,K] weight -> (values int8 [K/128,N,64], meta int32 [K/128,N,4] holding the
    uint32 index words): the 2:4 storage of include/w8a8.h (two largest |w| per group of 4)."""
    _check_tensor(wq, "wq", torch.int8, 2)
    N, K = wq.shape
    if values is None:
        values = _new((K // 128, N, 64), torch.int8, wq, stream)
    if meta is None:
        meta = _new((K // 128, N, 4), torch.int32, wq, stream)
    _check_tensor(values, "values", torch.int8, 3)
    _check_tensor(meta, "meta", torch.int32, 3)
    if tuple(values.shape) != (K // 128, N, 64) or tuple(meta.shape) != (K // 128, N, 4):
        raise ValueError("2:4 array shapes")
    _call("w8a8_compress24", wq.data_ptr(), N, K, values.data_ptr(), meta.data_ptr(),
          _stream_handle(stream))
    return values, meta


def w8a8_sparse24_gemm(xq, x_scale, values, meta, w_scale, out=None, out_dtype="bf16",
                       stream=None):
    """W8A8 GEMM on a compressed 2:4 weight (values [K/128,N,64] int8, meta [K/128,N,4] int32)."""
    od = _out_dtype(out_dtype)
    _check_tensor(xq, "xq", torch.int8, 2)
    _check_tensor(x_scale, "x_scale", torch.float32, 1)
    _check_tensor(values, "values", torch.int8, 3)
    _check_tensor(meta, "meta", torch.int32, 3)
    _check_tensor(w_scale, "w_scale", torch.float32, 1)
    M, K = xq.shape
    N = w_scale.shape[0]
    if (tuple(values.shape) != (K // 128, N, 64) or tuple(meta.shape) != (K // 128, N, 4)
            or tuple(x_scale.shape) != (M,)):
        raise ValueError("operand shapes")
    out = _out(out, M, N, od, xq, stream)
    _call("w8a8_sparse24_gemm", xq.data_ptr(), x_scale.data_ptr(), M, values.data_ptr(),
          meta.data_ptr(), w_scale.data_ptr(), N, K, out.data_ptr(), od, _stream_handle(stream))
    return out


def _w4a16_operands(wq4, scales, zeros):
    """Shapes and the 16-bit format (from the scales: bfloat16 or float16) of a W4A16 weight."""
    _check_tensor(wq4, "wq4", torch.uint8, 2)
    dt = scales.dtype if isinstance(scales, torch.Tensor) else None
    if dt not in (torch.bfloat16, torch.float16):
        raise TypeError("scales must be a bfloat16 or float16 tensor")
    _check_tensor(scales, "scales", dt, 2)
    _check_tensor(zeros, "zeros", dt, 2)
    N, K2 = wq4.shape
    K = 2 * K2
    if scales.shape != zeros.shape or scales.shape[0] != N or scales.shape[1] == 0 \
            or K % scales.shape[1]:
        raise ValueError("W4A16 operand shapes")
    return N, K, K // scales.shape[1], dt


W4A16_BF16, W4A16_F16 = 0, 1


def _w4a16_dtype(dt) -> int:
    return W4A16_F16 if dt == torch.float16 else W4A16_BF16


W4A16_CODES_U4, W4A16_CODES_S4 = 0, 1


def w4a16_dequant(wq4, scales, zeros, signed=False, out=None, stream=None):
    """Packed 4-bit codes [N,K/2] + scales/zeros [N,K/G] (bfloat16 or float16) -> w [N,K] of
    that type = round(round(q - z) * s); q the code (u4) or, with signed, its 4-bit two's
    complement (s4)."""
    N, K, G, dt = _w4a16_operands(wq4, scales, zeros)
    if out is None:
        out = _new((N, K), dt, wq4, stream)
    _check_tensor(out, "out", dt, 2)
    if tuple(out.shape) != (N, K):
        raise ValueError("out shape")
    _call("w4a16_dequant", wq4.data_ptr(), scales.data_ptr(), zeros.data_ptr(), N, K, G,
          W4A16_CODES_S4 if signed else W4A16_CODES_U4, _w4a16_dtype(dt), out.data_ptr(),
          _stream_handle(stream))
    return out


def w4a16_gemm(x, wq4, scales, zeros, signed=False, out=None, stream=None):
    """out [M,N] = x [M,K] times the dequantized 4-bit weights (u4, or s4 with signed), fused;
    x, scales, zeros and out all bfloat16 or all float16."""
    N, K, G, dt = _w4a16_operands(wq4, scales, zeros)
    _check_tensor(x, "x", dt, 2)
    M = x.shape[0]
    if x.shape[1] != K:
        raise ValueError("operand shapes")
    if out is None:
        out = _new((M, N), dt, x, stream)
    _check_tensor(out, "out", dt, 2)
    if tuple(out.shape) != (M, N):
        raise ValueError("out shape")
    _call("w4a16_gemm", x.data_ptr(), M, wq4.data_ptr(), scales.data_ptr(), zeros.data_ptr(), N,
          K, G, W4A16_CODES_S4 if signed else W4A16_CODES_U4, _w4a16_dtype(dt), out.data_ptr(),
          _stream_handle(stream))
    return out


def w8a8_bsr_gemm(xq, x_scale, crow, col, values, w_scale, out=None, out_dtype="bf16",
                  stream=None):
    """Block-sparse W8A8 GEMM; crow [N/64+1], col [nnzb], values [nnzb,64,64] int8."""
    od = _out_dtype(out_dtype)
    _check_tensor(xq, "xq", torch.int8, 2)
    _check_tensor(x_scale, "x_scale", torch.float32, 1)
    _check_tensor(crow, "crow", torch.int32, 1)
    _check_tensor(col, "col", torch.int32, 1)
    _check_tensor(values, "values", torch.int8, 3)
    _check_tensor(w_scale, "w_scale", torch.float32, 1)
    M, K = xq.shape
    nnzb, bs, bs2 = values.shape
    N = w_scale.shape[0]
    if bs != bs2 or col.shape[0] != nnzb or crow.shape[0] != N // max(bs, 1) + 1:
        raise ValueError("BSR array shapes")
    out = _out(out, M, N, od, xq, stream)
    _call("w8a8_bsr_gemm", xq.data_ptr(), x_scale.data_ptr(), M, K, crow.data_ptr(),
          col.data_ptr() if nnzb else 0, values.data_ptr() if nnzb else 0, nnzb, bs,
          w_scale.data_ptr(), N, out.data_ptr(), od, _stream_handle(stream))
    return out


def w8a8_bsr_gemm_addmm(xq, x_scale, crow, col, values, w_scale, bias=None, alpha=1.0, beta=None,
                        out=None, stream=None):
    """Block-sparse W8A8 GEMM with the addmm epilogue (bf16 out):
    out = bf16(alpha * (acc * x_scale[m] * w_scale[n]) + beta * bias[n]); bias None
    means no bias term; beta defaults to 1 with a bias and 0 without."""
    beta = _default_beta(bias, beta)
    _check_tensor(xq, "xq", torch.int8, 2)
    _check_tensor(x_scale, "x_scale", torch.float32, 1)
    _check_tensor(crow, "crow", torch.int32, 1)
    _check_tensor(col, "col", torch.int32, 1)
    _check_tensor(values, "values", torch.int8, 3)
    _check_tensor(w_scale, "w_scale", torch.float32, 1)
    M, K = xq.shape
    nnzb, bs, bs2 = values.shape
    N = w_scale.shape[0]
    if bs != bs2 or col.shape[0] != nnzb or crow.shape[0] != N // max(bs, 1) + 1:
        raise ValueError("BSR array shapes")
    if bias is not None:
        _check_tensor(bias, "bias", torch.float32, 1)
        if tuple(bias.shape) != (N,):
            raise ValueError("bias shape")
    out = _out(out, M, N, _out_dtype("bf16"), xq, stream)
    _call("w8a8_bsr_gemm_addmm", xq.data_ptr(), x_scale.data_ptr(), M, K, crow.data_ptr(),
          col.data_ptr() if nnzb else 0, values.data_ptr() if nnzb else 0, nnzb, bs,
          w_scale.data_ptr(), N, None if bias is None else bias.data_ptr(), float(alpha),
          float(beta), out.data_ptr(), _stream_handle(stream))
    return out


def w8a8_fused_linear(x, wq, w_scale, bias=None, alpha=1.0, beta=None, out=None, stream=None):
    """Single-launch quantize + GEMM for x [M,K] bf16 with M <= 64:
    out = bf16(alpha * (acc * s[m] * w_scale[n]) + beta * bias[n]), q and s as
    w8a8_quantize_rows computes them; bias None means no bias term; beta
    defaults to 1 with a bias and 0 without."""
    beta = _default_beta(bias, beta)
    _check_tensor(x, "x", torch.bfloat16, 2)
    _check_tensor(wq, "wq", torch.int8, 2)
    _check_tensor(w_scale, "w_scale", torch.float32, 1)
    M, K = x.shape
    N, K2 = wq.shape
    if K2 != K or tuple(w_scale.shape) != (N,):
        raise ValueError("operand shapes")
    if bias is not None:
        _check_tensor(bias, "bias", torch.float32, 1)
        if tuple(bias.shape) != (N,):
            raise ValueError("bias shape")
    out = _out(out, M, N, _out_dtype("bf16"), x, stream)
    _call("w8a8_fused_linear", x.data_ptr(), M, K, wq.data_ptr(), w_scale.data_ptr(), N,
          None if bias is None else bias.data_ptr(), float(alpha), float(beta), out.data_ptr(),
          _stream_handle(stream))
    return out


def w8a8_linear(x, wq, w_scale, out=None, stream=None):
    """Dynamically quantized linear layer: quantize_rows(x), then the fused-dequant GEMM.
    (Two launches are faster than w8a8_fused_linear at every M it takes: each of its
    N/16 workgroups quantizes all of x.)"""
    xq, xs = w8a8_quantize_rows(x, stream=stream)
    return w8a8_gemm(xq, xs, wq, w_scale, out=out, stream=stream)


# ---------------------------------------------------------------- MXFP4 and experts

MXFP4_BF16, MXFP4_F16, MXFP4_F32 = 0, 1, 2
MXFP4_MAX_K = 1048576
MOE_MAX_EXPERTS = 512
_MXFP4_DTYPES = {torch.bfloat16: MXFP4_BF16, torch.float16: MXFP4_F16, torch.float32: MXFP4_F32}


def _float_dtype(dtype, name="dtype") -> int:
    try:
        return _MXFP4_DTYPES[dtype]
    except (KeyError, TypeError):
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {dtype}") from None


# The entry points below are called once per layer and token while decoding, where the time of a
# call is the host's: a tensor that is as it should be passes one condition, the others go through
# _check_tensor for their message.

def _float_rows(t, name):
    """(dtype code, row stride, rows, width) of a 2-dim tensor of rows: its rows may lie apart."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _MXFP4_DTYPES.get(t.dtype)
    if code is None:
        code = _float_dtype(t.dtype, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dims, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    rows, width = t.shape
    if t.is_contiguous():
        return code, width, rows, width
    if width > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return code, t.stride(0) if rows > 1 else width, rows, width


def _check(t, name, dtype, ndim):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == ndim and t.is_cuda
            and t.is_contiguous()):
        _check_tensor(t, name, dtype, ndim)


def _result(t, name, shape, dtype, like, stream):
    """`t` checked, or a new tensor on `like`'s device."""
    if t is None:
        return _new(shape, dtype, like, stream)
    _check(t, name, dtype, len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _scratch(workspace, need, like, stream):
    """A workspace of `need` bytes: the caller's, or a new one. The caller of this function holds it
    until the library has been called: freed before the launch, its memory could go to another
    tensor that the kernels then write over."""
    if workspace is None:
        return _new((need,), torch.uint8, like, stream)
    _check(workspace, "workspace", torch.uint8, 1)
    return workspace


def _stream_of(t, stream) -> int:
    """The handle of `stream`, or of the current stream of t's device."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _done(st, fn):
    if st != W8A8_OK:
        raise W8A8Error(st, fn)


def _check_mx(codes, scales, names=("codes", "scales"), lead=()):
    """(rows, K) of MXFP4 rows: codes [*lead, rows, K/2], scales [*lead, ceil(K/256), rows, 8]."""
    n = len(lead)
    _check(codes, names[0], torch.uint8, 2 + n)
    _check(scales, names[1], torch.uint8, 3 + n)
    shape = codes.shape
    rows, K = shape[n], 2 * shape[n + 1]
    if shape[:n] != lead or scales.shape != lead + ((K + 255) // 256, rows, 8):
        raise ValueError(f"{names[1]} must have shape {lead + ((K + 255) // 256, rows, 8)} for "
                         f"{names[0]} {tuple(codes.shape)}, got {tuple(scales.shape)}")
    return rows, K


def mxfp4_quantize_rows(x, codes=None, scales=None, stream=None):
    """x [M,K] (bfloat16, float16 or float32; rows may lie apart) -> MXFP4: codes uint8 [M,K/2]
    and scales uint8 [ceil(K/256),M,8], the storage of include/w8a8.h."""
    dt, ld, M, K = _float_rows(x, "x")
    codes = _result(codes, "codes", (M, K // 2), torch.uint8, x, stream)
    scales = _result(scales, "scales", ((K + 255) // 256, M, 8), torch.uint8, x, stream)
    _done(load().mxfp4_quantize_rows(x.data_ptr(), ld, M, K, dt, codes.data_ptr(), scales.data_ptr(),
                                     _stream_of(x, stream)), "mxfp4_quantize_rows")
    return codes, scales


def mxfp4_dequantize_rows(codes, scales, dtype=torch.bfloat16, out=None, stream=None):
    """The values [M,K] that MXFP4 rows stand for, in `dtype`."""
    M, K = _check_mx(codes, scales)
    dt = _float_dtype(dtype)
    out = _result(out, "out", (M, K), dtype, codes, stream)
    _done(load().mxfp4_dequantize_rows(codes.data_ptr(), scales.data_ptr(), M, K, dt, out.data_ptr(),
                                       _stream_of(codes, stream)), "mxfp4_dequantize_rows")
    return out


def mxfp4_gemm(xq, xs, wq, ws, out=None, out_dtype=torch.bfloat16, stream=None):
    """out [M,N] = x times w transposed, both MXFP4 (xq [M,K/2], wq [N,K/2] and their scales)."""
    M, K = _check_mx(xq, xs, ("xq", "xs"))
    N, K2 = _check_mx(wq, ws, ("wq", "ws"))
    if K2 != K:
        raise ValueError("operand shapes")
    dt = _float_dtype(out_dtype, "out_dtype")
    out = _result(out, "out", (M, N), out_dtype, xq, stream)
    _done(load().mxfp4_gemm(xq.data_ptr(), xs.data_ptr(), M, wq.data_ptr(), ws.data_ptr(), N, K, dt,
                            out.data_ptr(), _stream_of(xq, stream)), "mxfp4_gemm")
    return out


def mxfp4_linear(x, wq, ws, out=None, out_dtype=None, workspace=None, stream=None):
    """out [M,N] = x [M,K], quantized to MXFP4 at run time, times the MXFP4 weight; out_dtype
    defaults to x's. workspace: uint8 of at least mxfp4_linear_workspace(M, N, K) bytes (a new
    one if None)."""
    xd, ld, M, K = _float_rows(x, "x")
    N, K2 = _check_mx(wq, ws, ("wq", "ws"))
    if K2 != K:
        raise ValueError("operand shapes")
    if out_dtype is None:
        out_dtype, od = x.dtype, xd
    else:
        od = _float_dtype(out_dtype, "out_dtype")
    lib = load()
    out = _result(out, "out", (M, N), out_dtype, x, stream)
    work, address, size = None, 0, 0
    need = lib.mxfp4_linear_workspace(M, N, K)
    if need or workspace is not None:
        work = _scratch(workspace, need, x, stream)
        address, size = work.data_ptr(), work.shape[0]
    _done(lib.mxfp4_linear(x.data_ptr(), ld, xd, M, wq.data_ptr(), ws.data_ptr(), N, K, od,
                           out.data_ptr(), address, size, _stream_of(x, stream)), "mxfp4_linear")
    return out


def mxfp4_linear_workspace(M, N, K) -> int:
    """Bytes of workspace that mxfp4_linear needs (0 for a few rows)."""
    return load().mxfp4_linear_workspace(M, N, K)


def _expert_ids(expert_ids):
    """(T, top, bits) of expert ids."""
    bits = {torch.int32: 32, torch.int64: 64}.get(getattr(expert_ids, "dtype", None))
    if bits is None:
        raise TypeError("expert_ids must be an int32 or int64 tensor")
    _check(expert_ids, "expert_ids", expert_ids.dtype, 2)
    T, top = expert_ids.shape
    return T, top, bits


def moe_sort(expert_ids, num_experts, offsets=None, slot_pos=None, row_token=None, workspace=None,
             stream=None):
    """Routing plan of expert_ids [T,top] (int32 or int64; ids outside [0, num_experts) are slots
    without an expert): (offsets int32 [num_experts+1], slot_pos int32 [T,top], row_token int32
    [T*top]) -- include/w8a8.h defines them. The order is stable."""
    T, top, bits = _expert_ids(expert_ids)
    offsets = _result(offsets, "offsets", (max(num_experts, 0) + 1,), torch.int32, expert_ids, stream)
    slot_pos = _result(slot_pos, "slot_pos", (T, top), torch.int32, expert_ids, stream)
    row_token = _result(row_token, "row_token", (T * top,), torch.int32, expert_ids, stream)
    lib = load()
    need = lib.moe_sort_workspace(T * top, num_experts)
    work, address, size = None, 0, 0
    if need or workspace is not None:
        work = _scratch(workspace, need, expert_ids, stream)
        address, size = work.data_ptr(), work.shape[0]
    _done(lib.moe_sort(expert_ids.data_ptr(), bits, T, top, num_experts, offsets.data_ptr(),
                       slot_pos.data_ptr(), row_token.data_ptr(), address, size,
                       _stream_of(expert_ids, stream)), "moe_sort")
    return offsets, slot_pos, row_token


def moe_sort_workspace(slots, num_experts) -> int:
    """Bytes of workspace that moe_sort needs for slots = T * top."""
    return load().moe_sort_workspace(slots, num_experts)


def moe_gather(x, slot_pos, out=None, stream=None):
    """Tokens x [T,H] -> rows [T*top,H] in expert order (0 for slots without an expert)."""
    dt, ld, T, H = _float_rows(x, "x")
    _check(slot_pos, "slot_pos", torch.int32, 2)
    top = slot_pos.shape[1]
    if slot_pos.shape[0] != T:
        raise ValueError("slot_pos must have a row per token")
    out = _result(out, "out", (T * top, H), x.dtype, x, stream)
    _done(load().moe_gather(x.data_ptr(), ld, slot_pos.data_ptr(), T, top, H, dt, out.data_ptr(),
                            _stream_of(x, stream)), "moe_gather")
    return out


def _sorted_rows(rows, name, slot_pos):
    """(dtype code, T, top, H) of rows in expert order with their plan."""
    code, _, n, H = _float_rows(rows, name)
    if not rows.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    _check(slot_pos, "slot_pos", torch.int32, 2)
    T, top = slot_pos.shape
    if n != T * top:
        raise ValueError(f"{name} must have a row per slot")
    return code, T, top, H


def moe_gather_backward(d_rows, slot_pos, out=None, stream=None):
    """Gradient of moe_gather: d_rows [T*top,H] -> d_x [T,H], the sum of each token's rows."""
    dt, T, top, H = _sorted_rows(d_rows, "d_rows", slot_pos)
    out = _result(out, "out", (T, H), d_rows.dtype, d_rows, stream)
    _done(load().moe_gather_backward(d_rows.data_ptr(), slot_pos.data_ptr(), T, top, H, dt,
                                     out.data_ptr(), _stream_of(d_rows, stream)),
          "moe_gather_backward")
    return out


def _routing_weights(weights, T, top):
    _check(weights, "weights", torch.float32, 2)
    if weights.shape != (T, top):
        raise ValueError("weights must have the shape of the routing")


def moe_combine(rows, slot_pos, weights, out=None, stream=None):
    """rows [T*top,H] in expert order -> out [T,H], each token's rows weighted by its router
    weights [T,top] (float32) and summed."""
    dt, T, top, H = _sorted_rows(rows, "rows", slot_pos)
    _routing_weights(weights, T, top)
    out = _result(out, "out", (T, H), rows.dtype, rows, stream)
    _done(load().moe_combine(rows.data_ptr(), slot_pos.data_ptr(), weights.data_ptr(), T, top, H, dt,
                             out.data_ptr(), _stream_of(rows, stream)), "moe_combine")
    return out


def moe_combine_backward(d_out, rows, slot_pos, weights, d_rows=None, d_weights=None, stream=None):
    """Gradients of moe_combine: d_out [T,H] -> (d_rows [T*top,H], d_weights float32 [T,top])."""
    dt, T, top, H = _sorted_rows(rows, "rows", slot_pos)
    _routing_weights(weights, T, top)
    dd, ld, n, width = _float_rows(d_out, "d_out")
    if dd != dt or n != T or width != H:
        raise ValueError("d_out must have the dtype of rows and a row per token")
    d_rows = _result(d_rows, "d_rows", (T * top, H), rows.dtype, rows, stream)
    d_weights = _result(d_weights, "d_weights", (T, top), torch.float32, rows, stream)
    _done(load().moe_combine_backward(d_out.data_ptr(), ld, rows.data_ptr(), slot_pos.data_ptr(),
                                      weights.data_ptr(), T, top, H, dt, d_rows.data_ptr(),
                                      d_weights.data_ptr(), _stream_of(rows, stream)),
          "moe_combine_backward")
    return d_rows, d_weights


def _expert_operands(xq, xs, offsets, wq, ws, row_token):
    """(T, S, E, N, K) of an experts' product."""
    T, K = _check_mx(xq, xs, ("xq", "xs"))
    if not isinstance(wq, torch.Tensor) or wq.dim() != 3:
        raise ValueError("wq must be a tensor [E, N, K/2]")
    E = wq.shape[0]
    N, K2 = _check_mx(wq, ws, ("wq", "ws"), (E,))
    _check(offsets, "offsets", torch.int32, 1)
    if K2 != K or offsets.shape[0] != E + 1:
        raise ValueError("operand shapes")
    if row_token is None:
        return T, T, E, N, K
    _check(row_token, "row_token", torch.int32, 1)
    return T, row_token.shape[0], E, N, K


def mxfp4_expert_gemm(xq, xs, offsets, wq, ws, row_token=None, out=None, out_dtype=torch.bfloat16,
                      stream=None):
    """out [S,N]: row r of expert e (offsets[e] <= r < offsets[e+1]) times weight e of wq [E,N,K/2],
    all MXFP4; rows past offsets[E] are 0. With row_token [S], row r is row row_token[r] of xq."""
    T, S, E, N, K = _expert_operands(xq, xs, offsets, wq, ws, row_token)
    dt = _float_dtype(out_dtype, "out_dtype")
    out = _result(out, "out", (S, N), out_dtype, xq, stream)
    _done(load().mxfp4_expert_gemm(xq.data_ptr(), xs.data_ptr(), T,
                                   None if row_token is None else row_token.data_ptr(), S,
                                   offsets.data_ptr(), E, wq.data_ptr(), ws.data_ptr(), N, K, dt,
                                   out.data_ptr(), _stream_of(xq, stream)), "mxfp4_expert_gemm")
    return out


def mxfp4_expert_swiglu(xq, xs, offsets, wq, ws, row_token=None, hq=None, hs=None, stream=None):
    """The experts' gate and up products (wq [E,2F,K/2], rows 2f the gate and 2f+1 the up
    projection of hidden unit f) and their SwiGLU, as MXFP4 rows (hq [S,F/2], hs)."""
    T, S, E, N, K = _expert_operands(xq, xs, offsets, wq, ws, row_token)
    F = N // 2
    if N % 64:
        raise ValueError("wq must have 2F rows per expert, F a multiple of 32")
    hq = _result(hq, "hq", (S, F // 2), torch.uint8, xq, stream)
    hs = _result(hs, "hs", ((F + 255) // 256, S, 8), torch.uint8, xq, stream)
    _done(load().mxfp4_expert_swiglu(xq.data_ptr(), xs.data_ptr(), T,
                                     None if row_token is None else row_token.data_ptr(), S,
                                     offsets.data_ptr(), E, wq.data_ptr(), ws.data_ptr(), F, K,
                                     hq.data_ptr(), hs.data_ptr(), _stream_of(xq, stream)),
          "mxfp4_expert_swiglu")
    return hq, hs


def mxfp4_moe(x, expert_ids, weights, w13q, w13s, w2q, w2s, out=None, workspace=None, stream=None):
    """An expert layer: x [T,H] quantized to MXFP4, routed by expert_ids [T,top] (int32 or int64)
    through the experts' gate/up weights w13 [E,2F,H] with SwiGLU and down weights w2 [E,H,F]
    (both MXFP4), and summed with the router's weights [T,top] (float32) -> out [T,H] of x's
    dtype. The experts' outputs and the sum are held in float32 and rounded once; a float16 layer
    of more than a few slots rounds the experts' outputs to float16's precision too. workspace:
    uint8 of at least mxfp4_moe_workspace(...) bytes (a new one if None)."""
    dt, ld, T, H = _float_rows(x, "x")
    T2, top, bits = _expert_ids(expert_ids)
    _routing_weights(weights, T, top)
    if not isinstance(w13q, torch.Tensor) or w13q.dim() != 3:
        raise ValueError("w13q must be a tensor [E, 2F, H/2]")
    E = w13q.shape[0]
    N, K = _check_mx(w13q, w13s, ("w13q", "w13s"), (E,))
    N2, F = _check_mx(w2q, w2s, ("w2q", "w2s"), (E,))
    if T2 != T or K != H or N2 != H or N != 2 * F:
        raise ValueError("operand shapes")
    lib = load()
    out = _result(out, "out", (T, H), x.dtype, x, stream)
    work = _scratch(workspace, lib.mxfp4_moe_workspace(T, top, E, H, F, dt), x, stream)
    _done(lib.mxfp4_moe(x.data_ptr(), ld, dt, T, H, expert_ids.data_ptr(), bits, weights.data_ptr(),
                        top, E, w13q.data_ptr(), w13s.data_ptr(), w2q.data_ptr(), w2s.data_ptr(), F,
                        out.data_ptr(), work.data_ptr(), work.shape[0], _stream_of(x, stream)), "mxfp4_moe")
    return out


def mxfp4_moe_workspace(T, top, num_experts, H, F, dtype=torch.bfloat16) -> int:
    """Bytes of workspace that mxfp4_moe needs."""
    return load().mxfp4_moe_workspace(T, top, num_experts, H, F, _float_dtype(dtype))


# ---------------------------------------------------------------- around a layer

W16A16_MAX_WIDTH = 1048576
BLOCK_NORM_MAX_H = 16384
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


def _activation(activation) -> int:
    code = ACTIVATIONS.get(activation) if isinstance(activation, str) else None
    if code is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {activation!r}")
    return code


def _vector(t, name, n):
    """The address of an fp32 vector [n], None for none."""
    if t is None:
        return None
    _check(t, name, torch.float32, 1)
    if t.shape[0] != n:
        raise ValueError(f"{name} must have shape {(n,)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _like_rows(t, name, dtype, shape):
    """(address, row stride) of rows of dtype and shape that may lie apart, (None, 0) for none."""
    if t is None:
        return None, 0
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.shape == shape:
        return t.data_ptr(), shape[1]
    _, ld, m, n = _float_rows(t, name)
    if t.dtype is not dtype or (m, n) != tuple(shape):
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, got {t.dtype} {(m, n)}")
    if ld < n:
        raise ValueError(f"{name} must have rows of their own, not expanded ones")
    return t.data_ptr(), ld


def _current(t, stream, *others):
    """The handle of `stream`, or of the current stream of t's device, on which every tensor has to be: a launch
    goes to the current device."""
    d = t.get_device()
    if d != torch._C._cuda_getDevice():
        raise ValueError(f"tensors are on cuda:{d}, the current device is cuda:{torch._C._cuda_getDevice()}")
    for o in others:
        if o is not None and o.get_device() != d:
            raise ValueError("all tensors must be on one device")
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(d)


def w8a8_gemm_act(xq, x_scale, wq, w_scale, bias=None, activation="none", residual=None, out=None,
                  stream=None):
    """out [M,N] = bf16(act(sum_k xq[m,k] wq[n,k] * x_scale[m] * w_scale[n] + bias[n]) + residual[m,n]);
    activation "none", "relu", "gelu", "gelu_tanh" or "silu"; bias float32 [N]; residual bfloat16 [M,N]
    (rows may lie apart), which may be `out` itself."""
    a = _activation(activation)
    _check(xq, "xq", torch.int8, 2)
    _check(x_scale, "x_scale", torch.float32, 1)
    _check(wq, "wq", torch.int8, 2)
    _check(w_scale, "w_scale", torch.float32, 1)
    M, K = xq.shape
    N, K2 = wq.shape
    if K2 != K or x_scale.shape[0] != M or w_scale.shape[0] != N:
        raise ValueError("operand shapes")
    b = _vector(bias, "bias", N)
    r, ldr = _like_rows(residual, "residual", torch.bfloat16, (M, N))
    s = _current(xq, stream, x_scale, wq, w_scale, bias, residual, out)
    out = _result(out, "out", (M, N), torch.bfloat16, xq, stream)
    _done(load().w8a8_gemm_act(xq.data_ptr(), x_scale.data_ptr(), M, wq.data_ptr(), w_scale.data_ptr(), N, K,
                               b, a, r, ldr, out.data_ptr(), s), "w8a8_gemm_act")
    return out


def _linear16_operands(x, w):
    """(dtype code, x's row stride, M, N, K) of 16-bit rows and their weight."""
    code, ld, M, K = _float_rows(x, "x")
    if code == MXFP4_F32:
        raise TypeError("x must be bfloat16 or float16")
    _check(w, "w", x.dtype, 2)
    N, K2 = w.shape
    if K2 != K:
        raise ValueError("operand shapes")
    return code, ld, M, N, K


def w16a16_linear(x, w, bias=None, activation="none", residual=None, pre=None, out=None, workspace=None,
                  stream=None):
    """out [M,N] = act(x w^T + bias) + residual for x [M,K] (rows may lie apart) and w [N,K], both bfloat16
    or both float16; bias float32 [N]; residual of x's dtype [M,N] (rows may lie apart), which may be `out`
    itself. pre: True or a tensor for x w^T + bias too, which the gradient of an activation needs; the result
    is (out, pre) then. workspace: uint8 of at least w16a16_linear_workspace(M, N, K) bytes (a new one if
    None); up to 16 rows a smaller one will do, in a longer time."""
    a = _activation(activation)
    code, ld, M, N, K = _linear16_operands(x, w)
    b = _vector(bias, "bias", N)
    r, ldr = _like_rows(residual, "residual", x.dtype, (M, N))
    if pre is False or pre is True:
        pre = _new((M, N), x.dtype, x, stream) if pre else None
    s = _current(x, stream, w, bias, residual, pre, out, workspace)
    p = None
    if pre is not None:
        p = _result(pre, "pre", (M, N), x.dtype, x, stream).data_ptr()
    out = _result(out, "out", (M, N), x.dtype, x, stream)
    lib = load()
    work, address, size = None, None, 0
    # (none at these sizes)
    need = 0 if M <= 16 and K <= 8192 and (N <= 4096 or K >= 1024) else lib.w16a16_linear_workspace(M, N, K)
    if need or workspace is not None:
        work = _scratch(workspace, need, x, stream)
        address, size = work.data_ptr(), work.shape[0]
    _done(lib.w16a16_linear(x.data_ptr(), ld, M, w.data_ptr(), N, K, code, b, a, r, ldr, p, out.data_ptr(),
                            address, size, s), "w16a16_linear")
    return out if pre is None else (out, pre)


def w16a16_linear_workspace(M, N, K) -> int:
    """Bytes of workspace that w16a16_linear needs (0 for most sizes)."""
    return load().w16a16_linear_workspace(M, N, K)


def _wanted(t, name, shape, dtype, like, stream):
    """A gradient: a new tensor for True, the caller's, or None for False or None (not wanted)."""
    if t is None or t is False:
        return None
    return _result(None if t is True else t, name, shape, dtype, like, stream)


def _address(t):
    return None if t is None else t.data_ptr()


def w16a16_linear_backward(d_out, x, w, pre=None, activation="none", d_x=True, d_w=True, d_bias=True,
                           d_pre=None, workspace=None, stream=None):
    """Gradients of w16a16_linear from d_out [M,N] (rows may lie apart) and, with an activation, the pre that it
    wrote: (d_x [M,K], d_w [N,K], d_bias float32 [N], d_pre [M,N]). d_x, d_w, d_bias: True for a new tensor,
    a tensor to write, False or None to leave it out (None in the result). d_pre = d_out act'(pre), rounded, is
    the operand of the products (d_out itself without an activation). The residual's gradient is d_out."""
    a = _activation(activation)
    code, ld, M, N, K = _linear16_operands(x, w)
    d, ldd = _like_rows(d_out, "d_out", x.dtype, (M, N))
    if d is None:
        raise TypeError("d_out must be a torch.Tensor")
    p = q = None
    if a:
        if pre is None:
            raise ValueError("the gradient of an activation needs pre")
        _check(pre, "pre", x.dtype, 2)
        if pre.shape != (M, N):
            raise ValueError(f"pre must have shape {(M, N)}, got {tuple(pre.shape)}")
        p = pre.data_ptr()
        d_pre = _result(d_pre, "d_pre", (M, N), x.dtype, x, stream)
        q = d_pre.data_ptr()
    else:
        pre, d_pre = None, d_out
    d_x = _wanted(d_x, "d_x", (M, K), x.dtype, x, stream)
    d_w = _wanted(d_w, "d_w", (N, K), x.dtype, x, stream)
    d_bias = _wanted(d_bias, "d_bias", (N,), torch.float32, x, stream)
    s = _current(x, stream, w, d_out, pre, d_pre, d_x, d_w, d_bias, workspace)
    lib = load()
    work, address, size = None, None, 0
    need = lib.w16a16_linear_backward_workspace(M, N, K)
    if need or workspace is not None:
        work = _scratch(workspace, need, x, stream)
        address, size = work.data_ptr(), work.shape[0]
    _done(lib.w16a16_linear_backward(d, ldd, x.data_ptr(), ld, w.data_ptr(), p, M, N, K, code, a, q, _address(d_x),
                                     _address(d_w), _address(d_bias), address, size, s), "w16a16_linear_backward")
    return d_x, d_w, d_bias, d_pre


def w16a16_linear_backward_workspace(M, N, K) -> int:
    """Bytes of workspace that w16a16_linear_backward needs."""
    return load().w16a16_linear_backward_workspace(M, N, K)


def _gate(gate, dtype, shape):
    """(address, row stride) of a gate: none, one float32 value per channel (stride 0), or rows."""
    if gate is None:
        return None, 0
    if isinstance(gate, torch.Tensor) and gate.dim() == 1:
        return _vector(gate, "gate", shape[1]), 0
    return _like_rows(gate, "gate", dtype, shape)


def _norm_operands(residual, weight, y, post_norm, post_weight, gate, scale, eps, new_residual, outputs, stream):
    """The library's arguments of a block norm up to its outputs, the new residual and the stream's handle."""
    code, ld, T, H = _float_rows(residual, "residual")
    dtype = residual.dtype
    w = _vector(weight, "weight", H)
    if y is None:
        if gate is not None or post_norm or post_weight is not None or new_residual is not None:
            raise ValueError("gate, post norm and new_residual need y")
        s = _current(residual, stream, weight, *outputs)
        return (residual.data_ptr(), ld, None, 0, 0, None, None, 0, scale, w, eps, T, H, code, None), residual, s
    y_at, ldy = _like_rows(y, "y", dtype, (T, H))
    gate_at, ldg = _gate(gate, dtype, (T, H))
    p = _vector(post_weight, "post_weight", H)
    s = _current(residual, stream, weight, y, post_weight, gate, new_residual, *outputs)
    new_residual = _result(new_residual, "new_residual", (T, H), dtype, residual, stream)
    return (residual.data_ptr(), ld, y_at, ldy, 1 if post_norm or post_weight is not None else 0, p, gate_at, ldg, scale, w,
            eps, T, H, code, new_residual.data_ptr()), new_residual, s


def block_norm(residual, weight=None, y=None, post_norm=False, post_weight=None, gate=None, scale=1.0, eps=1e-6,
               new_residual=None, out=None, stream=None):
    """The step between two blocks: (new_residual, out) with, per row,
    new_residual = residual + scale * gate * u, u = y or (post_norm, or a post_weight) y / rms(y) * post_weight,
    out = new_residual / rms(new_residual) * weight, rms(v) = sqrt(mean(v^2) + eps).
    residual, y: rows [T,H] of bfloat16, float16 or float32 (they may lie apart); gate: None, float32 [H], or
    rows; weight, post_weight: float32 [H] or None (ones). Without y it is the plain norm, and new_residual is
    residual. new_residual may be the (contiguous) residual or y."""
    args, new_residual, s = _norm_operands(residual, weight, y, post_norm, post_weight, gate, scale, eps, new_residual,
                                           (out,), stream)
    out = _result(out, "out", residual.shape, residual.dtype, residual, stream)
    _done(load().block_norm(*args, out.data_ptr(), s), "block_norm")
    return new_residual, out


def block_norm_w8a8(residual, weight=None, y=None, post_norm=False, post_weight=None, gate=None, scale=1.0,
                    eps=1e-6, new_residual=None, xq=None, x_scale=None, stream=None):
    """block_norm with its output quantized to int8 rows, as w8a8_quantize_rows would the unrounded output:
    (new_residual, xq int8 [T,H], x_scale float32 [T])."""
    args, new_residual, s = _norm_operands(residual, weight, y, post_norm, post_weight, gate, scale, eps, new_residual,
                                           (xq, x_scale), stream)
    xq = _result(xq, "xq", residual.shape, torch.int8, residual, stream)
    x_scale = _result(x_scale, "x_scale", residual.shape[:1], torch.float32, residual, stream)
    _done(load().block_norm_w8a8(*args, xq.data_ptr(), x_scale.data_ptr(), s), "block_norm_w8a8")
    return new_residual, xq, x_scale


def block_norm_mxfp4(residual, weight=None, y=None, post_norm=False, post_weight=None, gate=None, scale=1.0,
                     eps=1e-6, new_residual=None, codes=None, scales=None, stream=None):
    """block_norm with its output quantized to MXFP4 rows, as mxfp4_quantize_rows would the unrounded output:
    (new_residual, codes uint8 [T,H/2], scales uint8 [ceil(H/256),T,8])."""
    args, new_residual, s = _norm_operands(residual, weight, y, post_norm, post_weight, gate, scale, eps, new_residual,
                                           (codes, scales), stream)
    T, H = residual.shape
    codes = _result(codes, "codes", (T, H // 2), torch.uint8, residual, stream)
    scales = _result(scales, "scales", ((H + 255) // 256, T, 8), torch.uint8, residual, stream)
    _done(load().block_norm_mxfp4(*args, codes.data_ptr(), scales.data_ptr(), s), "block_norm_mxfp4")
    return new_residual, codes, scales


def block_norm_backward(d_out, new_residual, weight=None, d_residual=None, y=None, post_norm=False,
                        post_weight=None, gate=None, scale=1.0, eps=1e-6, workspace=None, stream=None):
    """Gradients of block_norm: d_out is out's, d_residual (rows, or None for 0) new_residual's, which is given as
    block_norm wrote it (without y: the residual). Returns (d_residual of the residual [T,H], d_weight float32 [H],
    d_y [T,H], d_post_weight float32 [H], d_gate [T,H] or float32 [H]), None for those without an input (the
    weights' gradients are given for absent weights, too, as those of ones; d_post_weight with a post norm)."""
    code, ldr, T, H = _float_rows(new_residual, "new_residual")
    dtype, shape = new_residual.dtype, (T, H)
    o, ldo = _like_rows(d_out, "d_out", dtype, shape)
    if o is None:
        raise TypeError("d_out must be a torch.Tensor")
    n, ldn = _like_rows(d_residual, "d_residual", dtype, shape)
    y_at, ldy = _like_rows(y, "y", dtype, shape)
    post = post_norm or post_weight is not None
    if y is None and (gate is not None or post):
        raise ValueError("gate and post norm need y")
    gate_at, ldg = _gate(gate, dtype, shape)
    w, p = _vector(weight, "weight", H), _vector(post_weight, "post_weight", H)
    s = _current(new_residual, stream, d_out, weight, d_residual, y, post_weight, gate, workspace)
    lib = load()
    d_r = _new(shape, dtype, new_residual, stream)
    d_weight = _new((H,), torch.float32, new_residual, stream)
    d_y = d_post_weight = d_gate = None
    if y is not None:
        d_y = _new(shape, dtype, new_residual, stream)
    if post:
        d_post_weight = _new((H,), torch.float32, new_residual, stream)
    if gate is not None:
        d_gate = _new(shape if ldg else (H,), dtype if ldg else torch.float32, new_residual, stream)
    work = _scratch(workspace, lib.block_norm_backward_workspace(T, H), new_residual, stream)
    _done(lib.block_norm_backward(o, ldo, n, ldn, new_residual.data_ptr(), ldr, y_at, ldy, 1 if post else 0, p, gate_at,
                                  ldg, scale, w, eps, T, H, code, d_r.data_ptr(), _address(d_y), _address(d_gate),
                                  d_weight.data_ptr(), _address(d_post_weight), work.data_ptr(), work.shape[0], s),
          "block_norm_backward")
    return d_r, d_weight, d_y, d_post_weight, d_gate


def block_norm_backward_workspace(T, H) -> int:
    """Bytes of workspace that block_norm_backward needs."""
    return load().block_norm_backward_workspace(T, H)
