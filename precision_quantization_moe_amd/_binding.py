"""ctypes binding of libpqmoe.so.  Argument marshalling only."""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpqmoe.so")

FMT_BF16, FMT_MXFP8, FMT_NVFP4, FMT_FP8_BLOCK = 0, 1, 2, 3
GEMM_FPROP, GEMM_DGRAD, GEMM_WGRAD = 0, 1, 2
OUT_BF16, OUT_FP32 = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
ACT_NONE, ACT_SILU, ACT_GELU = 0, 1, 2

_STATUS = {0: "ok", 1: "PQM_ERR_NULL", 2: "PQM_ERR_SHAPE", 3: "PQM_ERR_ALIGN",
           4: "PQM_ERR_ENUM", 5: "PQM_ERR_WORKSPACE", 6: "PQM_ERR_HIP"}


class PqmError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {_STATUS.get(code, code)}")
        self.code = code


_lib = None

P, I64, SZ, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
F32 = ctypes.c_float

# name -> argtypes; every entry point declared in include/pqmoe.h
SIGNATURES = {
    "pqm_status_string": ([I32], ctypes.c_char_p),
    "pqm_abi_version": ([], I32),
    "pqm_quantize_mxfp8": ([P, I64, I64, I64, P, P, P, P, P], I32),
    "pqm_quantize_fp8_block": ([P, I64, I64, I64, I64, P, P, P], I32),
    "pqm_quantize_nvfp4_per_token": ([P, I64, I64, I64, I64, P, P, P, P, SZ, P], I32),
    "pqm_quantize_nvfp4_workspace": ([I64, I64, I64], SZ),
    "pqm_dequantize": ([I32, P, P, P, I64, I64, I64, P, P], I32),
    "pqm_moe_grouped_gemm": ([I32, I32, P, P, P, P, P, P, I64, P, P, I64, I64, I64, I64,
                              P, I32, P, SZ, P], I32),
    "pqm_moe_grouped_gemm_workspace_size": ([I32, I32], SZ),
    "pqm_moe_fc2_online_nvfp4": ([P, P, P, P, I64, P, I64, I64, I64, I64, P, I32, P, P, P, P],
                                 I32),
    "pqm_moe_fc2_online_nvfp4_split": ([P, P, P, P, I64, P, I64, I64, I64, I64, P, I32, P, P, P,
                                        P, P], I32),
    "pqm_moe_gemm_swiglu_quantize_mxfp8": ([P, P, P, P, P, I64, I64, I64, I64, P, P, P, P, P],
                                           I32),
    "pqm_moe_route": ([P, I64, I64, I64, I32, P, P, P, P, P, SZ, P], I32),
    "pqm_moe_route_workspace": ([I64, I64, I64], SZ),
    "pqm_moe_route_noalloc": ([P, I64, I64, I64, I32, P, P, P, P, P], I32),
    "pqm_moe_gather_rows": ([P, I64, I64, P, I64, I64, P, P], I32),
    "pqm_moe_pad_rows": ([P, I64, I64, P, I64, I64, P, P, I64, P], I32),
    "pqm_swiglu_prob": ([P, P, P, I64, I64, P, P], I32),
    "pqm_swiglu_prob_quantize_mxfp8": ([P, P, P, I64, I64, P, P, P, P], I32),
    "pqm_swiglu_prob_quantize_nvfp4": ([P, P, P, I64, I64, P, P, P, P, P], I32),
    "pqm_moe_combine": ([P, P, P, I64, I64, I64, P, P], I32),
    "pqm_validate_offsets": ([P, I64, I64, I64, P, P], I32),
    "pqm_rmsnorm_quantize_mxfp8": ([P, I64, P, I64, P, I32, I64, I64, F32, P, P, P, P, P, P], I32),
    "pqm_rmsnorm_backward": ([P, P, P, I32, P, P, I64, I64, P, P, P, SZ, P], I32),
    "pqm_rmsnorm_backward_workspace": ([I64, I64], SZ),
    "pqm_moe_gate": ([P, I32, P, I64, I64, I64, I32, I32, F32, P, P, F32, P, P, P, P, SZ, P], I32),
    "pqm_moe_gate_workspace": ([I64, I64], SZ),
    "pqm_moe_gate_backward": ([P, I32, P, I64, I64, I64, I32, I32, F32, P, P, F32, P, P, P, I32,
                               P], I32),
    "pqm_moe_gemv_nvfp4": ([P, P, I64, I64, P, P, P, I64, I64, I64, I64, P, I32, P], I32),
    "pqm_moe_gemv_swiglu_nvfp4": ([P, P, P, I64, I64, P, P, P, I64, I64, I64, I64, P, P], I32),
    "pqm_linear": ([P, I64, P, P, I32, P, I64, I64, I64, I64, P, I32, P, P, SZ, P], I32),
    "pqm_linear_workspace": ([I64, I64, I64], SZ),
    "pqm_linear_backward": ([P, I64, P, I64, P, I32, P, P, I64, I64, I64, I64, P, P, P, P, P, SZ,
                             P], I32),
    "pqm_linear_backward_workspace": ([I64, I64, I64], SZ),
    "pqm_moe_decode_nvfp4": ([P, P, P, I32, F32, P, I64, I64, I64, I64, I64, I32, I32, I32, F32, P,
                              P, P, P, P, P, P, P, P, P, P, P, P, SZ, P], I32),
    "pqm_moe_decode_nvfp4_workspace": ([I64, I64, I64, I64, I64, I32], SZ),
    "pqm_token_logprobs": ([P, I32, I64, P, I64, I64, F32, P, P, P, P, P, I64, P, SZ, P], I32),
    "pqm_token_logprobs_workspace": ([I64, I64, I64], SZ),
    "pqm_token_logprobs_backward": ([P, I32, I64, P, I64, I64, F32, P, P, P, P, P, I32, I64, P],
                                    I32),
}


def lib():
    """Load libpqmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m precision_quantization_moe_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _check(code: int, what: str):
    if code != 0:
        raise PqmError(code, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


def _call(name: str, dev: torch.device, *args):
    """The entry point `name` on dev's current stream, with dev current: a
    kernel is launched on the current device.  (The raw stream getter takes a
    tenth of a microsecond; building a Stream object takes two, half the time
    of a launch.  The new tensors' sizes go to torch.empty as separate arguments
    for the same reason: 1.3 us instead of 1.7.)"""
    i = dev.index
    fn = getattr(_lib or lib(), name)
    stream = torch._C._cuda_getCurrentRawStream(i)
    if i == torch._C._cuda_getDevice():
        code = fn(*args, stream)
    else:
        with torch.cuda.device(i):
            code = fn(*args, stream)
    if code != 0:
        raise PqmError(code, name)


def _want(t: torch.Tensor, what: str, dtype, shape, dev: torch.device) -> torch.Tensor:
    """t, checked: a contiguous tensor of that type and shape on dev."""
    if t.dtype is not dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if t.device != dev:
        raise TypeError(f"{what}: on {t.device}, expected {dev}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    return t


def _bf16_or_f32(t: torch.Tensor, what: str) -> int:
    if t.dtype == torch.bfloat16:
        return OUT_BF16
    if t.dtype == torch.float32:
        return OUT_FP32
    raise TypeError(f"{what}: expected bfloat16 or float32, got {t.dtype}")


def _bf16_2d(x: torch.Tensor) -> torch.Tensor:
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise TypeError("expected a 2-D bfloat16 tensor")
    if not x.is_cuda:
        raise TypeError("expected a device tensor")
    if x.stride(1) != 1:
        raise ValueError("rows must be contiguous")
    return x


# ---------------------------------------------------------------- quantizers

def quantize_mxfp8(x: torch.Tensor, rowwise: bool = True, colwise: bool = True, out=None):
    """MXFP8 row-wise and/or column-wise copies of a bf16 [R, C] tensor.
    Returns (q[R, C], s[R, C/32], qT[C, R], sT[C, R/32]) as uint8 tensors,
    None for a copy that was not requested.  `out` may pass that tuple
    preallocated."""
    x = _bf16_2d(x)
    R, C = x.shape
    dev = x.device
    u8 = dict(dtype=torch.uint8, device=dev)
    if out is not None:
        q, s, qT, sT = out
    else:
        q = torch.empty((R, C), **u8) if rowwise else None
        s = torch.empty((R, C // 32), **u8) if rowwise else None
        qT = torch.empty((C, R), **u8) if colwise else None
        sT = torch.empty((C, R // 32), **u8) if colwise else None
    _check(lib().pqm_quantize_mxfp8(_ptr(x), R, C, x.stride(0), _ptr(q), _ptr(s),
                                    _ptr(qT), _ptr(sT), _stream(dev)),
           "pqm_quantize_mxfp8")
    return q, s, qT, sT


def quantize_fp8_block(x: torch.Tensor, block_rows: int = 1, out=None):
    """DeepSeek-style block FP8 of a bf16 [R, C] tensor: blocks of
    block_rows x 128 (1: activation tiles, 128: weight blocks).  Returns
    (q [R, C] uint8, s [R/block_rows, C/128] float32); `out` may pass them
    preallocated."""
    x = _bf16_2d(x)
    R, C = x.shape
    dev = x.device
    if out is not None:
        q, s = out
    else:
        q = torch.empty((R, C), dtype=torch.uint8, device=dev)
        s = torch.empty((R // block_rows, C // 128), dtype=torch.float32, device=dev)
    _check(lib().pqm_quantize_fp8_block(_ptr(x), R, C, x.stride(0), block_rows, _ptr(q),
                                        _ptr(s), _stream(dev)), "pqm_quantize_fp8_block")
    return q, s


def quantize_nvfp4_per_token(x: torch.Tensor, rows_per_scale: int = 1, out=None):
    """NVFP4 with one FP32 outer scale per rows_per_scale rows (1 = per
    token; an expert's [gate; up] row count = joint gate/up scale).
    Returns (q[R, C/2] uint8, s_block[R, C/16] uint8,
    s_outer[R/rows_per_scale] float32); `out` may pass them preallocated."""
    x = _bf16_2d(x)
    R, C = x.shape
    dev = x.device
    if out is not None:
        q, sb, sg = out
    else:
        q = torch.empty((R, C // 2), dtype=torch.uint8, device=dev)
        sb = torch.empty((R, C // 16), dtype=torch.uint8, device=dev)
        n_scales = R // rows_per_scale if rows_per_scale > 0 else 0
        sg = torch.empty((n_scales,), dtype=torch.float32, device=dev)
    L = lib()
    ws_bytes = L.pqm_quantize_nvfp4_workspace(R, C, rows_per_scale)
    ws = torch.empty((max(ws_bytes, 4),), dtype=torch.uint8, device=dev)
    _check(L.pqm_quantize_nvfp4_per_token(_ptr(x), R, C, x.stride(0), rows_per_scale,
                                          _ptr(q), _ptr(sb), _ptr(sg), _ptr(ws), ws_bytes,
                                          _stream(dev)),
           "pqm_quantize_nvfp4_per_token")
    return q, sb, sg


def dequantize(fmt: int, q: torch.Tensor, s_block: torch.Tensor,
               s_outer: torch.Tensor | None = None, rows_per_scale: int = 1, out=None):
    """bf16 [R, C] reconstruction of an MXFP8 or NVFP4 tensor."""
    R = q.shape[0]
    C = q.shape[1] * (2 if fmt == FMT_NVFP4 else 1)
    y = out if out is not None else torch.empty((R, C), dtype=torch.bfloat16, device=q.device)
    _check(lib().pqm_dequantize(fmt, _ptr(q), _ptr(s_block), _ptr(s_outer), R, C,
                                rows_per_scale, _ptr(y), _stream(q.device)),
           "pqm_dequantize")
    return y


# ---------------------------------------------------------------- norm

def rmsnorm_quantize_mxfp8(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                           residual: torch.Tensor | None = None, keep_y: bool = False,
                           quantize: bool = True, inplace: bool = False):
    """RMS norm of x (+ residual), its output encoded in MXFP8 row-wise; see
    pqm_rmsnorm_quantize_mxfp8 in pqmoe.h.  x, residual bf16 [R, C]; weight
    bf16 or float32 [C].  Returns (q, s, y, sum, rstd): q, s None without
    quantize; y (bf16) None unless keep_y or not quantize; sum = x + residual
    in bf16, x itself without a residual, and written into residual's memory
    with inplace; rstd float32 [R]."""
    x = _bf16_2d(x)
    R, C = x.shape
    dev = x.device
    wdt = _bf16_or_f32(weight, "weight")
    _want(weight, "weight", weight.dtype, (C,), dev)
    total = x
    if residual is not None:
        _bf16_2d(residual)
        if residual.shape != x.shape or residual.device != dev:
            raise ValueError("residual: expected x's shape and device")
        if inplace and not residual.is_contiguous():
            raise ValueError("residual: must be contiguous to be updated in place")
        total = residual if inplace else x.new_empty(R, C)
    q = s = y = None
    if quantize:
        q = torch.empty(R, C, dtype=torch.uint8, device=dev)
        s = torch.empty(R, C // 32, dtype=torch.uint8, device=dev)
    if keep_y or not quantize:
        y = x.new_empty(R, C)
    rstd = torch.empty(R, dtype=torch.float32, device=dev)
    _call("pqm_rmsnorm_quantize_mxfp8", dev, _ptr(x), x.stride(0) if R > 1 else C, _ptr(residual),
          residual.stride(0) if residual is not None and R > 1 else C, _ptr(weight), wdt, R, C,
          eps, None if residual is None else _ptr(total), _ptr(y), _ptr(q), _ptr(s), _ptr(rstd))
    return q, s, y, total, rstd


def rmsnorm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                     d_sum: torch.Tensor | None = None):
    """Gradients of rmsnorm_quantize_mxfp8; see pqm_rmsnorm_backward in
    pqmoe.h.  dy the gradient of y, x the forward call's sum, d_sum what
    reaches that sum past the norm.  Returns (dx bf16 [R, C], the gradient of
    x and of residual; dweight float32 [C])."""
    dy = _bf16_2d(dy)
    R, C = dy.shape
    dev = dy.device
    _want(dy, "dy", torch.bfloat16, (R, C), dev)
    _want(x, "x", torch.bfloat16, (R, C), dev)
    wdt = _bf16_or_f32(weight, "weight")
    _want(weight, "weight", weight.dtype, (C,), dev)
    _want(rstd, "rstd", torch.float32, (R,), dev)
    if d_sum is not None:
        _want(d_sum, "d_sum", torch.bfloat16, (R, C), dev)
    dx = x.new_empty(R, C)
    dw = torch.empty(C, dtype=torch.float32, device=dev)
    ws_bytes = lib().pqm_rmsnorm_backward_workspace(R, C)
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=dev)
    _call("pqm_rmsnorm_backward", dev, _ptr(dy), _ptr(x), _ptr(weight), wdt, _ptr(rstd),
          _ptr(d_sum), R, C, _ptr(dx), _ptr(dw), _ptr(ws), ws_bytes)
    return dx, dw


# ---------------------------------------------------------------- GEMM

def moe_grouped_gemm(fmt: int, kind: int, a, b, offsets: torch.Tensor, N: int, K: int,
                     a_scale=None, a_outer=None, b_scale=None, b_outer=None,
                     b_rows_per_scale: int = 0, out_dtype: int = OUT_FP32, out=None,
                     workspace: bool = True, bias=None):
    """Grouped GEMM over experts; see pqm_moe_grouped_gemm in pqmoe.h for the
    operand layouts.  offsets: int64 [G+1] on the device.  workspace=False
    passes none (the MXFP8 weight gradient then deals its tiles in a fixed
    order instead of handing them out).  bias: float32 [G, N] on the device
    (forward only), added in the epilogue."""
    G = offsets.numel() - 1
    # the MXFP8 weight gradient takes the transposed column-wise copies
    M = a.shape[1] if (fmt == FMT_MXFP8 and kind == GEMM_WGRAD) else a.shape[0]
    dev = offsets.device
    odt = torch.float32 if out_dtype == OUT_FP32 else torch.bfloat16
    if out is None:
        shape = (G, N, K) if kind == GEMM_WGRAD else (M, N)
        out = torch.empty(shape, dtype=odt, device=dev)
    L = lib()
    ws_bytes = L.pqm_moe_grouped_gemm_workspace_size(fmt, kind) if workspace else 0
    ws = torch.empty((max(ws_bytes, 16),), dtype=torch.uint8, device=dev) if ws_bytes else None
    _check(L.pqm_moe_grouped_gemm(fmt, kind, _ptr(a), _ptr(a_scale), _ptr(a_outer),
                                  _ptr(b), _ptr(b_scale), _ptr(b_outer),
                                  b_rows_per_scale, _ptr(bias), _ptr(offsets), G, M, N, K,
                                  _ptr(out), out_dtype, _ptr(ws), ws_bytes, _stream(dev)),
           "pqm_moe_grouped_gemm")
    return out


def moe_fc2_online_nvfp4(p: torch.Tensor, w_q, w_scale, w_outer, offsets: torch.Tensor, N: int,
                         w_rows_per_scale: int = 0, out_dtype: int = OUT_BF16,
                         encodings: bool = False):
    """NVFP4 down projection with online amax compensation; see
    pqm_moe_fc2_online_nvfp4 in pqmoe.h.  p: bf16 [M, K] device.  Returns
    (y, gs) or, with encodings, (y, gs, q, sb): the output, each row's final
    outer scale, and the codes / block scales P was encoded with."""
    G = offsets.numel() - 1
    M, K = p.shape
    dev = p.device
    odt = torch.float32 if out_dtype == OUT_FP32 else torch.bfloat16
    y = torch.empty((M, N), dtype=odt, device=dev)
    gs = torch.empty((M,), dtype=torch.float32, device=dev)
    q = torch.empty((M, K // 2), dtype=torch.uint8, device=dev) if encodings else None
    sb = torch.empty((M, K // 16), dtype=torch.uint8, device=dev) if encodings else None
    _check(lib().pqm_moe_fc2_online_nvfp4(_ptr(p), _ptr(w_q), _ptr(w_scale), _ptr(w_outer),
                                          w_rows_per_scale or N, _ptr(offsets), G, M, N, K,
                                          _ptr(y), out_dtype, _ptr(gs), _ptr(q), _ptr(sb),
                                          _stream(dev)),
           "pqm_moe_fc2_online_nvfp4")
    return (y, gs, q, sb) if encodings else (y, gs)


def moe_fc2_online_nvfp4_split(p: torch.Tensor, w_q, w_scale, w_outer, offsets: torch.Tensor,
                               N: int, w_rows_per_scale: int = 0, out_dtype: int = OUT_BF16,
                               encodings: bool = False):
    """The same FC2 split into two kernels (encode once, then the GEMM with
    the stored ratios); see pqm_moe_fc2_online_nvfp4_split in pqmoe.h.  The
    codes, block scales, gs and ratio buffers it needs are allocated here.
    Returns (y, gs) or, with encodings, (y, gs, q, sb, ratio)."""
    G = offsets.numel() - 1
    M, K = p.shape
    dev = p.device
    odt = torch.float32 if out_dtype == OUT_FP32 else torch.bfloat16
    y = torch.empty((M, N), dtype=odt, device=dev)
    gs = torch.empty((M,), dtype=torch.float32, device=dev)
    q = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    sb = torch.empty((M, K // 16), dtype=torch.uint8, device=dev)
    ratio = torch.empty((M, K // 128), dtype=torch.float32, device=dev)
    _check(lib().pqm_moe_fc2_online_nvfp4_split(_ptr(p), _ptr(w_q), _ptr(w_scale), _ptr(w_outer),
                                                w_rows_per_scale or N, _ptr(offsets), G, M, N, K,
                                                _ptr(y), out_dtype, _ptr(gs), _ptr(q), _ptr(sb),
                                                _ptr(ratio), _stream(dev)),
           "pqm_moe_fc2_online_nvfp4_split")
    return (y, gs, q, sb, ratio) if encodings else (y, gs)


_GEMV_TYPES = (torch.int32, torch.uint8, torch.uint8, torch.float32)


def _gemv_args(x, ids, rows_n, w_q, w_scale, w_outer, w_rows_per_scale, divisor):
    """Checked sizes of a few-row product: (rows, K, G, rows per scale) for
    weights of rows_n rows per expert."""
    K, dev, rows = _bf16_2d(x).shape[1], x.device, ids.numel()
    if divisor < 1 or rows_n < 1 or K < 32 or K % 32:
        raise PqmError(2, "pqm_moe_gemv_nvfp4")
    _want(x, "x", torch.bfloat16, (-(-rows // divisor), K), dev)
    if (ids.dtype, w_q.dtype, w_scale.dtype, w_outer.dtype) != _GEMV_TYPES or not (
            ids.device == w_q.device == w_scale.device == w_outer.device == dev):
        raise TypeError(f"expected ids int32, w_q and w_scale uint8, w_outer float32 on {dev}")
    if not (ids.is_contiguous() and w_q.is_contiguous() and w_scale.is_contiguous()
            and w_outer.is_contiguous()):
        raise ValueError("ids, w_q, w_scale, w_outer: must be contiguous")
    values = rows_n * (K // 2)
    G = w_q.numel() // values
    rps = w_rows_per_scale or rows_n
    if (w_q.numel() != G * values or 8 * w_scale.numel() != G * values
            or w_outer.numel() * rps != G * rows_n):
        raise ValueError("w_q, w_scale, w_outer: sizes do not belong together")
    return rows, K, G, rps


def moe_gemv_nvfp4(x: torch.Tensor, ids: torch.Tensor, w_q, w_scale, w_outer, N: int,
                   w_rows_per_scale: int = 0, divisor: int = 1, out_dtype: int = OUT_BF16):
    """A few routed rows times NVFP4 expert weights [G * N, K/2]; see
    pqm_moe_gemv_nvfp4 in pqmoe.h.  x bf16 [rows / divisor, K], ids int32 (any
    shape, one expert per row).  Returns [rows, N]."""
    rows, K, G, rps = _gemv_args(x, ids, N, w_q, w_scale, w_outer, w_rows_per_scale, divisor)
    dev = x.device
    odt = torch.float32 if out_dtype == OUT_FP32 else torch.bfloat16
    out = torch.empty(rows, N, dtype=odt, device=dev)
    _call("pqm_moe_gemv_nvfp4", dev, _ptr(x), _ptr(ids), rows, divisor, _ptr(w_q), _ptr(w_scale),
          _ptr(w_outer), rps, G, N, K, _ptr(out), out_dtype)
    return out


def moe_gemv_swiglu_nvfp4(x: torch.Tensor, ids: torch.Tensor, prob: torch.Tensor, w_q, w_scale,
                          w_outer, inter: int, w_rows_per_scale: int = 0, divisor: int = 1):
    """The gate_up product of a few routed rows with SwiGLU x prob in its
    epilogue, weights [G * 2 inter, K/2]; see pqm_moe_gemv_swiglu_nvfp4 in
    pqmoe.h.  prob float32, one per row.  Returns d bf16 [rows, inter]."""
    rows, K, G, rps = _gemv_args(x, ids, 2 * inter, w_q, w_scale, w_outer, w_rows_per_scale,
                                 divisor)
    dev = x.device
    _want(prob, "prob", torch.float32, prob.shape, dev)
    if prob.numel() != rows:
        raise ValueError("prob: expected one value per row")
    d = x.new_empty(rows, inter)
    _call("pqm_moe_gemv_swiglu_nvfp4", dev, _ptr(x), _ptr(ids), _ptr(prob), rows, divisor,
          _ptr(w_q), _ptr(w_scale), _ptr(w_outer), rps, G, inter, K, _ptr(d))
    return d


def moe_decode_nvfp4(x: torch.Tensor, residual: torch.Tensor | None, norm_w: torch.Tensor,
                     gate_w: torch.Tensor, w1_q, w1_scale, w1_outer, w2_q, w2_scale, w2_outer,
                     k: int, inter: int, shared: bool = False, score: int = SCORE_SOFTMAX,
                     renormalize: bool = True, scale: float = 1.0, eps: float = 1e-6):
    """A whole expert layer for up to 64 tokens, from the residual stream on; see
    pqm_moe_decode_nvfp4 in pqmoe.h.  x, residual (may be None) bf16 [T, H],
    norm_w bf16 or float32 [H], gate_w bf16 [E, H]; weights with one outer scale
    per expert, as moe_layer.quantize_expert_weights_nvfp4 returns them, of E
    experts, or of E + 1 with `shared`, whose last one every token meets.
    Returns (out [T, H], h [T, H], y [T, H] bf16, ids int32 and prob float32
    [T, k], d bf16 [T * (k + shared), inter])."""
    _bf16_2d(x)
    T, H = x.shape
    E, dev = gate_w.shape[0], x.device
    sh = 1 if shared else 0
    G = E + sh
    if inter < 0 or k < 1:
        raise PqmError(2, "pqm_moe_decode_nvfp4")
    _want(x, "x", torch.bfloat16, (T, H), dev)
    if residual is not None:
        _want(residual, "residual", torch.bfloat16, (T, H), dev)
    wdt = _bf16_or_f32(norm_w, "norm_w")
    _want(norm_w, "norm_w", norm_w.dtype, (H,), dev)
    _want(gate_w, "gate_w", torch.bfloat16, (E, H), dev)
    for name, t, dtype, n in (("w1_q", w1_q, torch.uint8, inter * H),
                              ("w1_scale", w1_scale, torch.uint8, inter * H // 8),
                              ("w1_outer", w1_outer, torch.float32, 1),
                              ("w2_q", w2_q, torch.uint8, H * inter // 2),
                              ("w2_scale", w2_scale, torch.uint8, H * inter // 16),
                              ("w2_outer", w2_outer, torch.float32, 1)):
        if t.dtype is not dtype or t.device != dev or not t.is_contiguous():
            raise TypeError(f"{name}: expected a contiguous {dtype} tensor on {dev}")
        if t.numel() != G * n:
            raise ValueError(f"{name}: expected {n} values for each of {G} experts, got {t.numel()}")
    size = lib().pqm_moe_decode_nvfp4_workspace(T, H, inter, E, k, sh)
    bf16 = dict(dtype=torch.bfloat16, device=dev)
    out, h, y = torch.empty(T, H, **bf16), torch.empty(T, H, **bf16), torch.empty(T, H, **bf16)
    ids = torch.empty(T, k, dtype=torch.int32, device=dev)
    prob = torch.empty(T, k, dtype=torch.float32, device=dev)
    d = torch.empty(T * (k + sh), inter, **bf16)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device=dev)
    _call("pqm_moe_decode_nvfp4", dev, _ptr(x), _ptr(residual), _ptr(norm_w), wdt, eps,
          _ptr(gate_w), T, H, inter, E, k, sh, score, int(renormalize), scale, _ptr(w1_q),
          _ptr(w1_scale), _ptr(w1_outer), _ptr(w2_q), _ptr(w2_scale), _ptr(w2_outer), _ptr(h),
          _ptr(y), _ptr(ids), _ptr(prob), _ptr(d), _ptr(out), _ptr(ws), size)
    return out, h, y, ids, prob, d


# ---------------------------------------------------------- dense products

def _rows(t: torch.Tensor, what: str, shape, dev: torch.device) -> int:
    """The row stride of t, a bf16 tensor of that shape on dev whose rows are
    contiguous."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{what}: expected torch.bfloat16, got {t.dtype}")
    if t.device != dev:
        raise TypeError(f"{what}: on {t.device}, expected {dev}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return shape[1]
    if t.stride(1) != 1 or t.stride(0) < shape[1]:
        raise ValueError(f"{what}: rows must be contiguous")
    return t.stride(0)


def linear(x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None = None,
           act: int = ACT_NONE, residual: torch.Tensor | None = None, keep_z: bool = False,
           out_dtype: int = OUT_BF16):
    """act(x w^T + bias) + residual in one pass; see pqm_linear in pqmoe.h.  x
    bf16 [M, K] and residual bf16 [M, N] with contiguous rows, w bf16 [N, K],
    bias float32 [N].  Returns (y [M, N], z bf16 [M, N]), z, what the activation
    took, None without keep_z."""
    _bf16_2d(x)
    M, K = x.shape
    N = w.shape[0]
    dev = x.device
    ldx = _rows(x, "x", (M, K), dev)
    _want(w, "w", torch.bfloat16, (N, K), dev)
    if bias is not None:
        _want(bias, "bias", torch.float32, (N,), dev)
    ldr = _rows(residual, "residual", (M, N), dev) if residual is not None else 0
    y = torch.empty(M, N, dtype=torch.float32 if out_dtype == OUT_FP32 else torch.bfloat16,
                    device=dev)
    z = torch.empty(M, N, dtype=torch.bfloat16, device=dev) if keep_z else None
    ws, size = None, 0
    if M > 64:
        size = lib().pqm_linear_workspace(M, N, K)
        if size:
            ws = torch.empty(size, dtype=torch.uint8, device=dev)
    _call("pqm_linear", dev, _ptr(x), ldx, _ptr(w), _ptr(bias), act, _ptr(residual), ldr, M, N, K,
          _ptr(y), out_dtype, _ptr(z), _ptr(ws), size)
    return y, z


def linear_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, act: int = ACT_NONE,
                    z: torch.Tensor | None = None, d_x: torch.Tensor | None = None,
                    need_dx: bool = True, need_dw: bool = True, need_dbias: bool = False):
    """Gradients of linear; see pqm_linear_backward in pqmoe.h.  dy bf16 [M, N]
    and x bf16 [M, K] with contiguous rows; z the forward call's, needed with an
    activation; d_x (bf16 [M, K], may be None): a gradient that reaches x past
    the product, added to dx.  Returns (dx bf16 [M, K], dw float32 [N, K],
    dbias float32 [N], dz bf16 [M, N]), None for what was not asked for; dz is
    None without an activation (it is dy)."""
    _bf16_2d(dy)
    M, N = dy.shape
    K = w.shape[1]
    dev = dy.device
    lddy = _rows(dy, "dy", (M, N), dev)
    ldx = _rows(x, "x", (M, K), dev)
    _want(w, "w", torch.bfloat16, (N, K), dev)
    dz = None
    if act != ACT_NONE:
        if z is None:
            raise ValueError("z: needed with an activation")
        _want(z, "z", torch.bfloat16, (M, N), dev)
        dz = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    ldd = _rows(d_x, "d_x", (M, K), dev) if d_x is not None else 0
    dx = torch.empty(M, K, dtype=torch.bfloat16, device=dev) if need_dx else None
    dw = torch.empty(N, K, dtype=torch.float32, device=dev) if need_dw else None
    db = torch.empty(N, dtype=torch.float32, device=dev) if need_dbias else None
    size = lib().pqm_linear_backward_workspace(M, N, K)
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
    _call("pqm_linear_backward", dev, _ptr(dy), lddy, _ptr(x), ldx, _ptr(w), act,
          _ptr(z) if act != ACT_NONE else None, _ptr(d_x), ldd, M, N, K, _ptr(dz), _ptr(dx),
          _ptr(dw), _ptr(db), _ptr(ws), size)
    return dx, dw, db, dz


# -------------------------------------------------------- log probabilities

def _logits(t: torch.Tensor, what: str):
    """(type, row stride) of logits [T, V] with contiguous rows."""
    dt = _bf16_or_f32(t, what)
    if not t.is_cuda:
        raise TypeError("expected a device tensor")
    if t.dim() != 2:
        raise ValueError(f"{what}: expected two dimensions")
    if t.is_contiguous():
        return dt, t.shape[1]
    if t.stride(1) != 1 or t.stride(0) < t.shape[1]:
        raise ValueError(f"{what}: rows must be contiguous")
    return dt, t.stride(0)


def token_logprobs(logits: torch.Tensor, ids: torch.Tensor | None = None,
                   temperature: float = 1.0, top_n: int = 0):
    """Log probabilities of given tokens, entropies and the best alternatives;
    see pqm_token_logprobs in pqmoe.h.  logits bf16 or float32 [T, V] with
    contiguous rows; ids int32 [T], negative for rows to leave out, None for
    alternatives alone.  Returns (logprob [T], entropy [T], stats [T, 2], top_ids
    int32 [T, top_n], top_logprob [T, top_n]), float32; logprob is None without
    ids, the last two without top_n."""
    dt, ld = _logits(logits, "logits")
    T, V = logits.shape
    dev = logits.device
    f32 = dict(dtype=torch.float32, device=dev)
    lp = None
    if ids is not None:
        _want(ids, "ids", torch.int32, (T,), dev)
        lp = torch.empty(T, **f32)
    entropy = torch.empty(T, **f32)
    stats = torch.empty(T, 2, **f32)
    top_ids = top_lp = ws = None
    if top_n:
        top_ids = torch.empty(T, max(top_n, 0), dtype=torch.int32, device=dev)
        top_lp = torch.empty(T, max(top_n, 0), **f32)
    size = lib().pqm_token_logprobs_workspace(T, V, top_n)
    if size:
        ws = torch.empty(size, dtype=torch.uint8, device=dev)
    _call("pqm_token_logprobs", dev, _ptr(logits), dt, ld, _ptr(ids), T, V, temperature, _ptr(lp),
          _ptr(entropy), _ptr(stats), _ptr(top_ids), _ptr(top_lp), top_n, _ptr(ws), size)
    return lp, entropy, stats, top_ids, top_lp


def token_logprobs_backward(logits: torch.Tensor, ids: torch.Tensor | None, stats: torch.Tensor,
                            d_logprob: torch.Tensor | None, temperature: float = 1.0,
                            entropy: torch.Tensor | None = None,
                            d_entropy: torch.Tensor | None = None, out_dtype: int | None = None,
                            out: torch.Tensor | None = None):
    """Gradient of token_logprobs with respect to its logits; see
    pqm_token_logprobs_backward in pqmoe.h.  stats and entropy are the forward
    call's (entropy with d_entropy alone).  Returns d_logits [T, V] in the
    logits' type unless out_dtype says otherwise; `out` may pass it, also the
    logits themselves."""
    dt, ld = _logits(logits, "logits")
    T, V = logits.shape
    dev = logits.device
    if ids is not None:
        _want(ids, "ids", torch.int32, (T,), dev)
    _want(stats, "stats", torch.float32, (T, 2), dev)
    for name, t in (("d_logprob", d_logprob), ("entropy", entropy), ("d_entropy", d_entropy)):
        if t is not None:
            _want(t, name, torch.float32, (T,), dev)
    odt = dt if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty(T, V, dtype=torch.float32 if odt == OUT_FP32 else torch.bfloat16,
                          device=dev)
        ldd = V
    else:
        odt, ldd = _logits(out, "out")
        if out.shape != logits.shape or out.device != dev:
            raise ValueError("out: expected the logits' shape and device")
    _call("pqm_token_logprobs_backward", dev, _ptr(logits), dt, ld, _ptr(ids), T, V, temperature,
          _ptr(stats), _ptr(entropy), _ptr(d_logprob), _ptr(d_entropy), _ptr(out), odt, ldd)
    return out


# ---------------------------------------------------------------- MoE glue

def moe_gate(logits: torch.Tensor, k: int, score: int = SCORE_SOFTMAX, renormalize: bool = True,
             scale: float = 1.0, mask: torch.Tensor | None = None,
             loss_coef: float | None = None):
    """The router's gate; see pqm_moe_gate in pqmoe.h.  logits bf16 or float32
    [T, E]; mask uint8 or bool [T], zero for tokens to leave out.  Returns
    (topk_ids int32 [T, k], prob float32 [T, k], counts int32 [E + 1],
    prob_sum float32 [E], loss float32 [1]), the last three None without a
    loss_coef."""
    T, E = logits.shape
    dev = logits.device
    zdt = _bf16_or_f32(logits, "logits")
    if not logits.is_cuda:
        raise TypeError("expected a device tensor")
    _want(logits, "logits", logits.dtype, (T, E), dev)
    if mask is not None:
        _want(mask, "mask", torch.bool if mask.dtype == torch.bool else torch.uint8, (T,), dev)
    ids = torch.empty(T, max(k, 0), dtype=torch.int32, device=dev)
    prob = torch.empty(T, max(k, 0), dtype=torch.float32, device=dev)
    counts = prob_sum = loss = ws = None
    ws_bytes = 0
    if loss_coef is not None:
        counts = torch.empty(E + 1, dtype=torch.int32, device=dev)
        prob_sum = torch.empty(E, dtype=torch.float32, device=dev)
        loss = torch.empty(1, dtype=torch.float32, device=dev)
        ws_bytes = lib().pqm_moe_gate_workspace(T, E)
        ws = torch.empty(max(ws_bytes, 4), dtype=torch.uint8, device=dev)
    _call("pqm_moe_gate", dev, _ptr(logits), zdt, _ptr(mask), T, E, k, score, int(renormalize),
          scale, _ptr(ids), _ptr(prob), loss_coef or 0.0, _ptr(counts), _ptr(prob_sum), _ptr(loss),
          _ptr(ws), ws_bytes)
    return ids, prob, counts, prob_sum, loss


def moe_gate_backward(logits: torch.Tensor, ids: torch.Tensor, d_prob: torch.Tensor | None,
                      score: int = SCORE_SOFTMAX, renormalize: bool = True, scale: float = 1.0,
                      mask: torch.Tensor | None = None, loss_coef: float | None = None,
                      counts: torch.Tensor | None = None, d_loss: torch.Tensor | None = None,
                      out_dtype: int | None = None):
    """Gradient of moe_gate with respect to its logits; see
    pqm_moe_gate_backward in pqmoe.h.  d_prob float32 [T, k] or None; counts
    the forward call's and d_loss float32 [1], or both None.  Returns d_logits
    [T, E], in the logits' type unless out_dtype says otherwise."""
    T, E = logits.shape
    dev = logits.device
    zdt = _bf16_or_f32(logits, "logits")
    if not logits.is_cuda:
        raise TypeError("expected a device tensor")
    _want(logits, "logits", logits.dtype, (T, E), dev)
    k = ids.shape[-1]
    _want(ids, "ids", torch.int32, (T, k), dev)
    if d_prob is not None:
        _want(d_prob, "d_prob", torch.float32, (T, k), dev)
    if mask is not None:
        _want(mask, "mask", torch.bool if mask.dtype == torch.bool else torch.uint8, (T,), dev)
    if counts is not None:
        _want(counts, "counts", torch.int32, (E + 1,), dev)
        if loss_coef is None:
            raise ValueError("counts: needs the forward call's loss_coef")
    if d_loss is not None:
        _want(d_loss, "d_loss", torch.float32, d_loss.shape, dev)
        if d_loss.numel() != 1:
            raise ValueError("d_loss: expected one value")
    odt = zdt if out_dtype is None else out_dtype
    dz = torch.empty(T, E, dtype=torch.float32 if odt == OUT_FP32 else torch.bfloat16,
                     device=dev)
    _call("pqm_moe_gate_backward", dev, _ptr(logits), zdt, _ptr(mask), T, E, k, score,
          int(renormalize), scale, _ptr(ids), _ptr(d_prob), loss_coef or 0.0, _ptr(counts),
          _ptr(d_loss), _ptr(dz), odt)
    return dz


def moe_route(topk_ids: torch.Tensor, num_experts: int, shared_expert: bool = False):
    """Counting sort of assignments by expert.  topk_ids int32 [T, k].
    Returns (offsets int64 [E+1(+1)], src_row int32 [M], token int32 [M],
    slot int32 [T, k]) with M = T*k (+T with a shared expert group)."""
    T, k = topk_ids.shape
    dev = topk_ids.device
    sh = 1 if shared_expert else 0
    M = T * k + sh * T
    offsets = torch.empty((num_experts + 1 + sh,), dtype=torch.int64, device=dev)
    src = torch.empty((M,), dtype=torch.int32, device=dev)
    tok = torch.empty((M,), dtype=torch.int32, device=dev)
    slot = torch.empty((T, k), dtype=torch.int32, device=dev)
    L = lib()
    ws_bytes = L.pqm_moe_route_workspace(T, k, num_experts)
    ws = torch.empty((max(ws_bytes, 4),), dtype=torch.uint8, device=dev)
    _check(L.pqm_moe_route(_ptr(topk_ids), T, k, num_experts, sh, _ptr(offsets), _ptr(src),
                           _ptr(tok), _ptr(slot), _ptr(ws), ws_bytes, _stream(dev)),
           "pqm_moe_route")
    return offsets, src, tok, slot


def moe_route_noalloc(topk_ids: torch.Tensor, num_experts: int, shared_expert: bool = False,
                      out=None):
    """moe_route through the entry point that allocates nothing on the
    device: its scratch is the library's per-GPU array.  `out` may pass the
    (offsets, src_row, token, slot) tensors preallocated, so that the call
    itself allocates nothing."""
    T, k = topk_ids.shape
    dev = topk_ids.device
    sh = 1 if shared_expert else 0
    M = T * k + sh * T
    if out is None:
        out = (torch.empty((num_experts + 1 + sh,), dtype=torch.int64, device=dev),
               torch.empty((M,), dtype=torch.int32, device=dev),
               torch.empty((M,), dtype=torch.int32, device=dev),
               torch.empty((T, k), dtype=torch.int32, device=dev))
    offsets, src, tok, slot = out
    _check(lib().pqm_moe_route_noalloc(_ptr(topk_ids), T, k, num_experts, sh, _ptr(offsets),
                                       _ptr(src), _ptr(tok), _ptr(slot), _stream(dev)),
           "pqm_moe_route_noalloc")
    return offsets, src, tok, slot


def moe_gather_rows(src: torch.Tensor, index: torch.Tensor, divisor: int = 1):
    """out[i] = src[index[i] // divisor] for a 2-D byte-addressable tensor."""
    n = index.numel()
    out = torch.empty((n,) + tuple(src.shape[1:]), dtype=src.dtype, device=src.device)
    row_bytes = src.stride(0) * src.element_size()
    _check(lib().pqm_moe_gather_rows(_ptr(src), src.shape[0], row_bytes, _ptr(index), n,
                                     divisor, _ptr(out), _stream(src.device)),
           "pqm_moe_gather_rows")
    return out


def pad_rows_bound(rows: int, groups: int, align: int = 32) -> int:
    """Rows that any per-expert padding of `rows` rows in `groups` groups
    fits in, rounded up to a whole block."""
    n = rows + groups * (align - 1)
    return -(-n // align) * align


def moe_pad_rows(src: torch.Tensor, offsets: torch.Tensor, align: int = 32, out=None,
                 padded_offsets=None):
    """Each group's rows of a 2-D tensor moved to a start that is a multiple
    of `align`, padding rows zero.  Returns (out [pad_rows_bound(...), ...],
    padded_offsets int64 [G+1] on the device)."""
    G = offsets.numel() - 1
    rows = src.shape[0]
    if out is None:
        out = torch.empty((pad_rows_bound(rows, G, align),) + tuple(src.shape[1:]),
                          dtype=src.dtype, device=src.device)
    if padded_offsets is None:
        padded_offsets = torch.empty(G + 1, dtype=torch.int64, device=src.device)
    row_bytes = src.stride(0) * src.element_size()
    _check(lib().pqm_moe_pad_rows(_ptr(src), rows, row_bytes, _ptr(offsets), G, align,
                                  _ptr(padded_offsets), _ptr(out), out.shape[0],
                                  _stream(src.device)), "pqm_moe_pad_rows")
    return out, padded_offsets


def swiglu_prob(c: torch.Tensor, prob: torch.Tensor, src: torch.Tensor | None = None):
    """D = silu(gate) * up * prob per row, gate/up the two halves of c.
    prob float32 indexed by src[row] (flat assignment index) when given."""
    M, N2 = c.shape
    d = torch.empty((M, N2 // 2), dtype=torch.bfloat16, device=c.device)
    _check(lib().pqm_swiglu_prob(_ptr(c), _ptr(prob), _ptr(src), M, N2 // 2, _ptr(d),
                                 _stream(c.device)), "pqm_swiglu_prob")
    return d


def swiglu_prob_quantize_mxfp8(c: torch.Tensor, prob: torch.Tensor,
                               src: torch.Tensor | None = None, keep_d: bool = False):
    """swiglu_prob fused with the row-wise MXFP8 quantization of its output.
    Returns (q, s, d) with d None unless keep_d."""
    M, N2 = c.shape
    inter = N2 // 2
    q = torch.empty((M, inter), dtype=torch.uint8, device=c.device)
    s = torch.empty((M, inter // 32), dtype=torch.uint8, device=c.device)
    d = torch.empty((M, inter), dtype=torch.bfloat16, device=c.device) if keep_d else None
    _check(lib().pqm_swiglu_prob_quantize_mxfp8(_ptr(c), _ptr(prob), _ptr(src), M, inter,
                                                _ptr(d), _ptr(q), _ptr(s), _stream(c.device)),
           "pqm_swiglu_prob_quantize_mxfp8")
    return q, s, d


def swiglu_prob_quantize_nvfp4(c: torch.Tensor, prob: torch.Tensor,
                               src: torch.Tensor | None = None, keep_d: bool = False):
    """swiglu_prob fused with the per-token NVFP4 quantization of its output.
    Returns (q, s_block, s_outer, d) with d None unless keep_d."""
    M, N2 = c.shape
    inter = N2 // 2
    dev = c.device
    q = torch.empty((M, inter // 2), dtype=torch.uint8, device=dev)
    sb = torch.empty((M, inter // 16), dtype=torch.uint8, device=dev)
    sg = torch.empty((M,), dtype=torch.float32, device=dev)
    d = torch.empty((M, inter), dtype=torch.bfloat16, device=dev) if keep_d else None
    _check(lib().pqm_swiglu_prob_quantize_nvfp4(_ptr(c), _ptr(prob), _ptr(src), M, inter, _ptr(d),
                                                _ptr(q), _ptr(sb), _ptr(sg), _stream(dev)),
           "pqm_swiglu_prob_quantize_nvfp4")
    return q, sb, sg, d


def moe_gemm_swiglu_quantize_mxfp8(qa, sa, w1q, w1s, offsets: torch.Tensor, inter: int,
                                   prob: torch.Tensor, src: torch.Tensor | None = None):
    """MXFP8 gate_up grouped GEMM with SwiGLU x prob and the row-wise MXFP8
    quantization of D fused into its epilogue.  Returns (qd, sd)."""
    G = offsets.numel() - 1
    M, K = qa.shape
    q = torch.empty((M, inter), dtype=torch.uint8, device=qa.device)
    s = torch.empty((M, inter // 32), dtype=torch.uint8, device=qa.device)
    _check(lib().pqm_moe_gemm_swiglu_quantize_mxfp8(
        _ptr(qa), _ptr(sa), _ptr(w1q), _ptr(w1s), _ptr(offsets), G, M, inter, K, _ptr(prob),
        _ptr(src), _ptr(q), _ptr(s), _stream(qa.device)), "pqm_moe_gemm_swiglu_quantize_mxfp8")
    return q, s


def moe_combine(y_rows: torch.Tensor, slot: torch.Tensor, shared: torch.Tensor | None = None):
    """out[t] = sum_j y_rows[slot[t, j]] (+ shared[t]), bf16 output."""
    T, k = slot.shape
    N = y_rows.shape[1]
    out = torch.empty((T, N), dtype=torch.bfloat16, device=y_rows.device)
    _check(lib().pqm_moe_combine(_ptr(y_rows), _ptr(slot), _ptr(shared), T, k, N, _ptr(out),
                                 _stream(y_rows.device)), "pqm_moe_combine")
    return out


OFFSETS_FIRST_NOT_ZERO, OFFSETS_DECREASING, OFFSETS_MISALIGNED, OFFSETS_PAST_END = 1, 2, 3, 4


def validate_offsets(offsets: torch.Tensor, M_total: int, align: int = 1):
    """Opt-in check of an offsets array (int64 [G+1] on the device) against
    the grouped-GEMM contract.  Returns an int32 device tensor [2]: (first
    failing check or 0, its index or -1); see pqm_validate_offsets."""
    G = offsets.numel() - 1
    res = torch.empty((2,), dtype=torch.int32, device=offsets.device)
    _check(lib().pqm_validate_offsets(_ptr(offsets), G, M_total, align, _ptr(res),
                                      _stream(offsets.device)),
           "pqm_validate_offsets")
    return res
