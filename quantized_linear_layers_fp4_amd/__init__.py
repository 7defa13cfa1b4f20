"""MI355X (gfx950) FP4 quantized linear-layer forward: Python binding of libfp4lin.so.

Argument marshalling only: torch supplies device memory and the current HIP stream,
and every step of the forward runs in the library's HIP kernels (include/fp4lin.h is
the ABI).  There is no CPU fallback: without the built library every call raises.

    Y = linear_forward(A, W, q)            # A: M x K, W: K x N (cuda, bf16 or fp32)

The method (quantization of A per token and W per output channel into E2M1, outlier
clamping at a quantile of |A| with sparse compensation dA) follows the pages on
"Optimizing Large Language Model Training Using FP4 Quantization" (QbitAI report:
granularity, forward-quantization and outlier paragraphs).
"""
from __future__ import annotations

import ctypes as C
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp4lin.so")

FP4_F32, FP4_BF16 = 0, 1
FP4_Q16 = 2  # fp4_gemm output only: int16 4*acc with fp32 escapes in the workspace
FP4_PER_ROW, FP4_PER_COL = 0, 1
FP4_STAGE_A, FP4_STAGE_W = 1, 2
FP4_BLOCK_VECTOR, FP4_BLOCK_SQUARE = 0, 1

EXPORTS = (
    "fp4_quantize", "fp4_outlier_capacity", "fp4_outlier_workspace_bytes", "fp4_outlier_clamp",
    "fp4_outlier_clamp_noalloc",
    "fp4_gemm_workspace_bytes", "fp4_gemm", "fp4_forward_layout", "fp4_forward_workspace_bytes", "fp4_linear_forward",
    "fp4_linear_forward_wq", "fp4_forward_quantize", "fp4_forward_product", "fp4_gemm_fp8emu_workspace_bytes", "fp4_gemm_fp8emu",
    "fp4_fp8_workspace_bytes", "fp4_fp8_quantize", "fp4_fp8_dequantize",
    "fp4_backward_layout", "fp4_backward_workspace_bytes", "fp4_linear_backward",
    "fp4_block8_codes_bytes", "fp4_block8_scales_bytes", "fp4_block8_quantize", "fp4_block8_dequantize",
    "fp4_block8_gemm", "fp4_block8_linear_workspace_bytes", "fp4_block8_linear",
    "fp4_block8_backward_workspace_bytes", "fp4_block8_backward",
    "fp4_kv4_cache_bytes", "fp4_kv4_write", "fp4_kv4_read", "fp4_kv4_attention_workspace_bytes", "fp4_kv4_attention",
    "fp4_kv4_attention_sinks", "fp4_kv4_attention_shared_parts", "fp4_kv4_attention_shared_workspace_bytes", "fp4_kv4_attention_shared",
    "fp4_kv4_extend_workspace_bytes", "fp4_kv4_extend", "fp4_kv4_release_workspace_bytes", "fp4_kv4_release",
    "fp4_rope_table", "fp4_qk_norm_rope", "fp4_kv4_norm_rope", "fp4_qk_norm_rope_backward_workspace_bytes",
    "fp4_qk_norm_rope_backward",
    "fp4_gemm_kernel_name", "fp4_comp_kernel_name", "fp4_status_string",
)


class WsLayout(C.Structure):
    _fields_ = [(n, C.c_size_t) for n in ("total", "T", "nnz", "row_ptr", "coo_row", "coo_col", "coo_val",
                                          "Aq", "sA", "Wq", "sW", "handoff", "scratch")] + [("capacity", C.c_int64)]


class BwdLayout(C.Structure):
    _fields_ = [(n, C.c_size_t) for n in ("total", "Gq", "sG", "Hq", "sH", "WqT", "AqT", "ones", "part")]


class Fp4Error(RuntimeError):
    pass


_lib = None


def lib():
    """Load libfp4lin.so from the package directory (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise Fp4Error(f"{LIB_PATH} is missing: build it with `python -m quantized_linear_layers_fp4_amd.build`")
    L = C.CDLL(LIB_PATH)
    vp, i64, i32, dbl, sz = C.c_void_p, C.c_int64, C.c_int32, C.c_double, C.c_size_t
    sig = {
        "fp4_quantize": (i32, [vp, i32, i64, i64, i32, vp, vp, vp, vp]),
        "fp4_outlier_capacity": (i64, [i64, i64, dbl]),
        "fp4_outlier_workspace_bytes": (sz, [i64, i64, i32, dbl]),
        "fp4_outlier_clamp": (i32, [vp, i32, i64, i64, dbl, vp, vp, vp, vp, i64, vp, vp, vp, sz, vp]),
        "fp4_outlier_clamp_noalloc": (i32, [vp, i32, i64, i64, dbl, vp, vp, vp, vp, i64, vp, vp, vp]),
        "fp4_gemm_workspace_bytes": (sz, [i64, i64, i32, i32]),
        "fp4_gemm": (i32, [vp, vp, vp, vp, i64, i64, i64, vp, vp, vp, i64, vp, i32, vp, i32, vp, vp, sz, vp]),
        "fp4_forward_layout": (i32, [i64, i64, i64, i32, i32, dbl, C.POINTER(WsLayout)]),
        "fp4_forward_workspace_bytes": (sz, [i64, i64, i64, i32, i32, dbl]),
        "fp4_linear_forward": (i32, [vp, vp, i32, i64, i64, i64, dbl, vp, i32, vp, sz, vp]),
        "fp4_linear_forward_wq": (i32, [vp, vp, vp, vp, i32, i64, i64, i64, dbl, vp, i32, vp, sz, vp]),
        "fp4_forward_quantize": (i32, [vp, vp, i32, i64, i64, i64, dbl, i32, vp, sz, vp]),
        "fp4_forward_product": (i32, [vp, i32, i64, i64, i64, dbl, vp, i32, vp, sz, vp]),
        "fp4_gemm_fp8emu_workspace_bytes": (sz, [i64, i64, i64]),
        "fp4_fp8_workspace_bytes": (sz, []),
        "fp4_fp8_quantize": (i32, [vp, i32, i64, vp, vp, vp, sz, vp]),
        "fp4_fp8_dequantize": (i32, [vp, i64, vp, vp, i32, vp]),
        "fp4_gemm_fp8emu": (i32, [vp, vp, vp, vp, i64, i64, i64, vp, i32, vp, vp, sz, vp]),
        "fp4_backward_layout": (i32, [i64, i64, i64, C.POINTER(BwdLayout)]),
        "fp4_backward_workspace_bytes": (sz, [i64, i64, i64]),
        "fp4_linear_backward": (i32, [vp, i32, i64, i64, i64, vp, vp, vp, vp, vp, i32, vp, i32, vp, sz, vp]),
        "fp4_block8_codes_bytes": (sz, [i64, i64]),
        "fp4_block8_scales_bytes": (sz, [i64, i64, i32]),
        "fp4_block8_quantize": (i32, [vp, i32, i64, i64, i64, i32, vp, vp, vp, vp, vp]),
        "fp4_block8_dequantize": (i32, [vp, vp, i64, i64, i32, vp, i32, vp]),
        "fp4_block8_gemm": (i32, [vp, vp, i32, vp, vp, i32, i64, i64, i64, vp, i32, vp]),
        "fp4_block8_linear_workspace_bytes": (sz, [i64, i64, i64]),
        "fp4_block8_linear": (i32, [vp, i32, i64, i64, i64, vp, vp, i32, i64, vp, i32, vp, vp, vp, sz, vp]),
        "fp4_block8_backward_workspace_bytes": (sz, [i64, i64]),
        "fp4_block8_backward": (i32, [vp, i32, i64, i64, i64, i64, vp, vp, i32, vp, vp, vp, i32, vp, i32, vp, sz, vp]),
        "fp4_kv4_cache_bytes": (sz, [i64, i32, i32, i32]),
        "fp4_kv4_write": (i32, [vp, i64, i32, i32, i32, vp, vp, i32, i64, i64, i64, i64, i64, vp, i32, vp]),
        "fp4_kv4_read": (i32, [vp, i64, i32, i32, i32, vp, i32, i64, vp, vp, i32, vp]),
        "fp4_kv4_attention_workspace_bytes": (sz, [i32, i32, i32, i32, i32, i32, i32]),
        "fp4_kv4_attention": (i32, [vp, i64, i64, i64, i32, vp, vp, i32, i32, vp, i64, i32, vp, i64, i32, i32, i32,
                                    i32, C.c_float, vp, vp, vp, sz, vp]),
        "fp4_kv4_attention_sinks": (i32, [vp, i64, i64, i64, i32, vp, vp, i32, i32, vp, i64, i32, vp, i64, i32, i32, i32,
                                          i32, i32, C.c_float, vp, vp, vp, sz, vp]),
        "fp4_kv4_attention_shared_parts": (i32, [i64, i32, i32, i32, i32, i32, i32, i32, i32]),
        "fp4_kv4_attention_shared_workspace_bytes": (sz, [i64, i32, i32, i32, i32, i32, i32, i32, i32]),
        "fp4_kv4_attention_shared": (i32, [vp, i64, i64, i64, i32, vp, vp, i32, i32, vp, i64, i32, vp, i64, i32, i32, i32,
                                           i32, C.c_float, vp, vp, vp, sz, vp]),
        "fp4_kv4_extend_workspace_bytes": (sz, [i32, i64]),
        "fp4_kv4_extend": (i32, [vp, i64, i32, i32, vp, vp, vp, i64, i32, vp, i64, vp, vp, vp, vp, sz, vp]),
        "fp4_kv4_release_workspace_bytes": (sz, [i32, i32]),
        "fp4_kv4_release": (i32, [vp, i64, i32, i32, vp, vp, vp, i64, i32, vp, i32, i32, i32, vp, sz, vp]),
        "fp4_rope_table": (i32, [vp, i64, i32, dbl, dbl, vp]),
        "fp4_qk_norm_rope": (i32, [vp, i64, i64, i32, vp, i64, i64, i32, i64, i32, i32, vp, vp, i32, C.c_float, vp, vp, i64,
                                   i32, i32, vp, vp, vp]),
        "fp4_kv4_norm_rope": (i32, [vp, i64, i32, vp, i64, i64, i32, vp, i64, i64, vp, i64, i64, i32, i64, i32, i32, vp, i32,
                                    vp, vp, i32, C.c_float, vp, vp, i64, i32, i32, vp, vp]),
        "fp4_qk_norm_rope_backward_workspace_bytes": (sz, [i32]),
        "fp4_qk_norm_rope_backward": (i32, [vp, i64, i64, vp, i64, i64, vp, i64, i64, i32, vp, i64, i64, i32, i64, i32, i32,
                                            vp, vp, i32, C.c_float, vp, vp, i64, i32, i32, vp, i64, i64, vp, i64, i64, vp,
                                            vp, vp, sz, vp]),
        "fp4_gemm_kernel_name": (C.c_char_p, [i64, i64, i64, i32]),
        "fp4_comp_kernel_name": (C.c_char_p, [i64, i64]),
        "fp4_status_string": (C.c_char_p, [i32]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    _lib = L
    return L


def _check(status: int):
    if status != 0:
        raise Fp4Error(f"fp4 status {status}: {lib().fp4_status_string(status).decode()}")


_DT_CODE = {torch.bfloat16: FP4_BF16, torch.float32: FP4_F32}


def _dt(t: torch.Tensor) -> int:
    code = _DT_CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"expected bfloat16 or float32, got {t.dtype}")
    return code


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _stream(t: torch.Tensor):
    # the current stream's handle without a Stream object around it (0.1 against 2.1 us a call)
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous and on a HIP device")


def _out_dtype_code(d: torch.dtype) -> int:
    return _DT_CODE[d]


# --------------------------------------------------------------------------- calls
def quantize(X: torch.Tensor, axis: int = FP4_PER_ROW, clamp_T: torch.Tensor | None = None):
    """E2M1 codes and fp32 scales of X (R x C).  PER_ROW: codes R x C/2, scales R.
    PER_COL: codes C x R/2 (transposed), scales C."""
    _need_cuda(X, clamp_T)
    R, Cn = X.shape
    if axis == FP4_PER_ROW:
        codes = torch.empty((R, Cn // 2), dtype=torch.uint8, device=X.device)
        scales = torch.empty(R, dtype=torch.float32, device=X.device)
    else:
        codes = torch.empty((Cn, R // 2), dtype=torch.uint8, device=X.device)
        scales = torch.empty(Cn, dtype=torch.float32, device=X.device)
    _check(lib().fp4_quantize(_ptr(X), _dt(X), R, Cn, axis, _ptr(clamp_T), _ptr(codes), _ptr(scales), _stream(X)))
    return codes, scales


def gemm_kernel_name(M: int, N: int, K: int, num_cus: int) -> str:
    """The FP4 GEMM kernel the library launches for an M x N x K product on num_cus CUs."""
    r = lib().fp4_gemm_kernel_name(M, N, K, num_cus)
    if r is None:
        raise Fp4Error(f"no GEMM kernel for M={M} N={N} K={K} on {num_cus} CUs")
    return r.decode()


def comp_kernel_name(M: int, capacity: int) -> str:
    """The compensation kernel the library launches for M rows and a dA list of `capacity`."""
    r = lib().fp4_comp_kernel_name(M, capacity)
    if r is None:
        raise Fp4Error(f"no compensation kernel for M={M} capacity={capacity}")
    return r.decode()


def outlier_capacity(M: int, K: int, q: float) -> int:
    return int(lib().fp4_outlier_capacity(M, K, float(q)))


def outlier_clamp(A: torch.Tensor, q: float, trim: bool = True) -> dict:
    """Threshold T and the COO list of dA for A (M x K).  With trim=True the COO arrays
    are cut to nnz (this reads nnz back and synchronizes)."""
    _need_cuda(A)
    M, K = A.shape
    L = lib()
    cap = int(L.fp4_outlier_capacity(M, K, float(q)))
    if cap < 0:
        _check(2)
    dev = A.device
    capn = max(cap, 1)
    T = torch.empty(4, dtype=torch.float32, device=dev)
    coo_row = torch.empty(capn, dtype=torch.int32, device=dev)
    coo_col = torch.empty(capn, dtype=torch.int32, device=dev)
    coo_val = torch.empty(capn, dtype=torch.float32, device=dev)
    row_ptr = torch.empty(M + 1, dtype=torch.int32, device=dev)
    nnz = torch.empty(2, dtype=torch.int64, device=dev)
    wsb = int(L.fp4_outlier_workspace_bytes(M, K, _dt(A), float(q)))
    ws = torch.empty(wsb, dtype=torch.uint8, device=dev)
    _check(L.fp4_outlier_clamp(_ptr(A), _dt(A), M, K, float(q), _ptr(T), _ptr(coo_row), _ptr(coo_col),
                               _ptr(coo_val), capn, _ptr(row_ptr), _ptr(nnz), _ptr(ws), wsb, _stream(A)))
    out = dict(T=T[:1], row_ptr=row_ptr, nnz=nnz[:1], coo_row=coo_row, coo_col=coo_col, coo_val=coo_val)
    if trim:
        n = int(nnz[0].item())
        out.update(coo_row=coo_row[:n], coo_col=coo_col[:n], coo_val=coo_val[:n])
    return out


def gemm(Aq: torch.Tensor, sA: torch.Tensor, Wq: torch.Tensor, sW: torch.Tensor, K: int,
         row_ptr: torch.Tensor | None = None, coo_col: torch.Tensor | None = None,
         coo_val: torch.Tensor | None = None, W: torch.Tensor | None = None,
         out_dtype: torch.dtype = torch.bfloat16, acc_out: bool = False, ws: torch.Tensor | None = None,
         capacity: int | None = None):
    """Y = fl(fl(acc * sA) * sW) (+ dA . W when row_ptr, coo_col, coo_val and W are given)."""
    _need_cuda(Aq, sA, Wq, sW, row_ptr, coo_col, coo_val, W, ws)
    M, N = Aq.shape[0], Wq.shape[0]
    Y = torch.empty((M, N), dtype=out_dtype, device=Aq.device)
    acc = torch.empty((M, N), dtype=torch.float32, device=Aq.device) if acc_out else None
    wdt = _dt(W) if W is not None else FP4_BF16
    with_comp = int(row_ptr is not None and coo_col is not None and coo_val is not None)
    if ws is None:
        nbytes = lib().fp4_gemm_workspace_bytes(M, N, _out_dtype_code(out_dtype), with_comp)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=Aq.device) if nbytes else None
    cap = capacity if capacity is not None else (coo_col.numel() if coo_col is not None else 0)
    _check(lib().fp4_gemm(_ptr(Aq), _ptr(sA), _ptr(Wq), _ptr(sW), M, N, K, _ptr(row_ptr), _ptr(coo_col),
                          _ptr(coo_val), cap, _ptr(W), wdt, _ptr(Y), _out_dtype_code(out_dtype), _ptr(acc), _ptr(ws),
                          ws.numel() if ws is not None else 0, _stream(Aq)))
    return (Y, acc) if acc_out else Y


def gemm_q16(Aq: torch.Tensor, sA: torch.Tensor, Wq: torch.Tensor, sW: torch.Tensor, K: int,
             acc_out: bool = False):
    """The exact accumulator in two bytes (FP4_Q16): (Yq int16 M x N, esc fp32 M x N), where
    Yq = 4*acc, except in the escaped 128 x 64 blocks (those around some |acc| > 8191.75):
    there Yq = -32768 and esc = fl(fl(acc*sA)*sW)."""
    _need_cuda(Aq, sA, Wq, sW)
    M, N = Aq.shape[0], Wq.shape[0]
    Yq = torch.empty((M, N), dtype=torch.int16, device=Aq.device)
    acc = torch.empty((M, N), dtype=torch.float32, device=Aq.device) if acc_out else None
    nbytes = lib().fp4_gemm_workspace_bytes(M, N, FP4_Q16, 0)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=Aq.device)
    _check(lib().fp4_gemm(_ptr(Aq), _ptr(sA), _ptr(Wq), _ptr(sW), M, N, K, None, None, None, 0, None, FP4_BF16,
                          _ptr(Yq), FP4_Q16, _ptr(acc), _ptr(ws), nbytes, _stream(Aq)))
    esc = ws[:M * N * 4].view(torch.float32).view(M, N)  # the escape values come first in the workspace
    return (Yq, esc, acc) if acc_out else (Yq, esc)


def gemm_fp8emu(Aq: torch.Tensor, sA: torch.Tensor, Wq: torch.Tensor, sW: torch.Tensor, K: int,
                out_dtype: torch.dtype = torch.bfloat16, acc_out: bool = False, ws: torch.Tensor | None = None):
    """The product on E4M3 matrix cores after an exact E2M1 -> E4M3 expansion (no dA term)."""
    _need_cuda(Aq, sA, Wq, sW, ws)
    M, N = Aq.shape[0], Wq.shape[0]
    Y = torch.empty((M, N), dtype=out_dtype, device=Aq.device)
    acc = torch.empty((M, N), dtype=torch.float32, device=Aq.device) if acc_out else None
    if ws is None:
        nbytes = lib().fp4_gemm_fp8emu_workspace_bytes(M, N, K)
        if nbytes == 0:
            raise Fp4Error("shape out of range for the FP8 emulation")
        ws = torch.empty(nbytes, dtype=torch.uint8, device=Aq.device)
    _check(lib().fp4_gemm_fp8emu(_ptr(Aq), _ptr(sA), _ptr(Wq), _ptr(sW), M, N, K, _ptr(Y), _out_dtype_code(out_dtype),
                                 _ptr(acc), _ptr(ws), ws.numel(), _stream(Aq)))
    return (Y, acc) if acc_out else Y


def fp8_quantize(X: torch.Tensor):
    """FP8 (E4M3) gradient codec: (codes u8[n], scale fp32[1]) with one per-tensor scale."""
    _need_cuda(X)
    n = X.numel()
    codes = torch.empty(n, dtype=torch.uint8, device=X.device)
    scale = torch.empty(1, dtype=torch.float32, device=X.device)
    ws = torch.empty(lib().fp4_fp8_workspace_bytes(), dtype=torch.uint8, device=X.device)
    _check(lib().fp4_fp8_quantize(_ptr(X), _dt(X), n, _ptr(codes), _ptr(scale), _ptr(ws), ws.numel(), _stream(X)))
    return codes, scale


def fp8_dequantize(codes: torch.Tensor, scale: torch.Tensor, out_dtype: torch.dtype = torch.float32):
    _need_cuda(codes, scale)
    Y = torch.empty(codes.numel(), dtype=out_dtype, device=codes.device)
    _check(lib().fp4_fp8_dequantize(_ptr(codes), codes.numel(), _ptr(scale), _ptr(Y), _out_dtype_code(out_dtype),
                                    _stream(codes)))
    return Y


def forward_layout(M: int, K: int, N: int, dtype: torch.dtype, q: float,
                   out_dtype: torch.dtype | None = None) -> WsLayout:
    """The forward workspace's layout for inputs of dtype and Y of out_dtype (default: dtype)."""
    lay = WsLayout()
    _check(lib().fp4_forward_layout(M, K, N, _out_dtype_code(dtype), _out_dtype_code(out_dtype or dtype), float(q),
                                    C.byref(lay)))
    return lay


def workspace(A: torch.Tensor, N: int, q: float, out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """A workspace tensor sized for linear_forward(A, W (K x N), q, out_dtype)."""
    M, K = A.shape
    lay = forward_layout(M, K, N, A.dtype, q, out_dtype)
    return torch.empty(lay.total, dtype=torch.uint8, device=A.device)


def linear_forward(A: torch.Tensor, W: torch.Tensor, q: float, out_dtype: torch.dtype | None = None,
                   ws: torch.Tensor | None = None, Y: torch.Tensor | None = None) -> torch.Tensor:
    """FP4 linear forward Y = dequant(Aq . Wq) + dA . W on the current stream."""
    _need_cuda(A, W, ws, Y)
    if A.dtype != W.dtype:
        raise TypeError("A and W must share a dtype")
    M, K = A.shape
    N = W.shape[1]
    out_dtype = out_dtype or A.dtype
    if ws is None:
        ws = workspace(A, N, q, out_dtype)
    if Y is None:
        Y = torch.empty((M, N), dtype=out_dtype, device=A.device)
    _check(lib().fp4_linear_forward(_ptr(A), _ptr(W), _dt(A), M, K, N, float(q), _ptr(Y), _dt(Y), _ptr(ws),
                                    ws.numel(), _stream(A)))
    return Y


def forward_quantize(A: torch.Tensor | None, W: torch.Tensor | None, M: int, K: int, N: int, dtype: torch.dtype,
                     q: float, ws: torch.Tensor, stages: int = FP4_STAGE_A | FP4_STAGE_W):
    """The forward's quantizer stages (FP4_STAGE_A and/or FP4_STAGE_W) into the workspace."""
    _need_cuda(A, W, ws)
    dt = FP4_BF16 if dtype == torch.bfloat16 else FP4_F32
    ref = A if A is not None else W
    _check(lib().fp4_forward_quantize(_ptr(A), _ptr(W), dt, M, K, N, float(q), stages, _ptr(ws), ws.numel(),
                                      _stream(ref)))


def forward_product(W: torch.Tensor, M: int, q: float, ws: torch.Tensor, Y: torch.Tensor):
    """The forward's product stage (GEMM, dequantization, compensation) from the workspace."""
    _need_cuda(W, ws, Y)
    K, N = W.shape
    _check(lib().fp4_forward_product(_ptr(W), _dt(W), M, K, N, float(q), _ptr(Y), _dt(Y), _ptr(ws), ws.numel(),
                                     _stream(W)))
    return Y


def quantize_weights(W: torch.Tensor):
    """(Wq, sW) of a K x N weight matrix: per-output-channel codes (N x K/2) and scales."""
    _need_cuda(W)
    K, N = W.shape
    Wq = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device)
    sW = torch.empty(N, dtype=torch.float32, device=W.device)
    _check(lib().fp4_quantize(_ptr(W), _dt(W), K, N, FP4_PER_COL, None, _ptr(Wq), _ptr(sW), _stream(W)))
    return Wq, sW


def linear_forward_wq(A: torch.Tensor, W: torch.Tensor, Wq: torch.Tensor, sW: torch.Tensor, q: float,
                      out_dtype: torch.dtype | None = None, ws: torch.Tensor | None = None,
                      Y: torch.Tensor | None = None) -> torch.Tensor:
    """The forward with W's codes and scales from quantize_weights(W) (W unchanged since)."""
    _need_cuda(A, W, Wq, sW, ws, Y)
    if A.dtype != W.dtype:
        raise TypeError("A and W must share a dtype")
    M, K = A.shape
    N = W.shape[1]
    out_dtype = out_dtype or A.dtype
    if ws is None:
        ws = workspace(A, N, q, out_dtype)
    if Y is None:
        Y = torch.empty((M, N), dtype=out_dtype, device=A.device)
    _check(lib().fp4_linear_forward_wq(_ptr(A), _ptr(W), _ptr(Wq), _ptr(sW), _dt(A), M, K, N, float(q), _ptr(Y),
                                       _dt(Y), _ptr(ws), ws.numel(), _stream(A)))
    return Y


def forward_intermediates(ws: torch.Tensor, M: int, K: int, N: int, dtype: torch.dtype, q: float) -> dict:
    """Views of T, nnz, the COO list, codes and scales inside a forward workspace."""
    lay = forward_layout(M, K, N, dtype, q)
    cap = max(int(lay.capacity), 1)

    def view(off, count, dt, shape=None):
        nbytes = count * torch.tensor([], dtype=dt).element_size()
        t = ws[off:off + nbytes].view(dt)
        return t.view(shape) if shape else t

    return dict(
        T=view(lay.T, 1, torch.float32), nnz=view(lay.nnz, 1, torch.int64),
        row_ptr=view(lay.row_ptr, M + 1, torch.int32), coo_row=view(lay.coo_row, cap, torch.int32),
        coo_col=view(lay.coo_col, cap, torch.int32), coo_val=view(lay.coo_val, cap, torch.float32),
        Aq=view(lay.Aq, M * (K // 2), torch.uint8, (M, K // 2)), sA=view(lay.sA, M, torch.float32),
        Wq=view(lay.Wq, N * (K // 2), torch.uint8, (N, K // 2)), sW=view(lay.sW, N, torch.float32),
        capacity=int(lay.capacity))


# --------------------------------------------------------------------------- backward
def backward_layout(M: int, K: int, N: int) -> BwdLayout:
    lay = BwdLayout()
    _check(lib().fp4_backward_layout(M, K, N, C.byref(lay)))
    return lay


def linear_backward(dY: torch.Tensor, Aq: torch.Tensor | None, sA: torch.Tensor | None, Wq: torch.Tensor | None,
                    sW: torch.Tensor | None, K: int, want_dA: bool = True, want_dW: bool = True,
                    out_dtype: torch.dtype | None = None, ws: torch.Tensor | None = None,
                    dA: torch.Tensor | None = None, dW: torch.Tensor | None = None):
    """Straight-through backward of the quantized product: (dA, dW), each None when not
    wanted.  Aq/sA/Wq/sW are the forward's codes and scales (forward_intermediates)."""
    _need_cuda(dY, Aq, sA, Wq, sW, ws, dA, dW)
    M, N = dY.shape
    out_dtype = out_dtype or dY.dtype
    if ws is None:
        ws = torch.empty(backward_layout(M, K, N).total, dtype=torch.uint8, device=dY.device)
    if want_dA and dA is None:
        dA = torch.empty((M, K), dtype=out_dtype, device=dY.device)
    if want_dW and dW is None:
        dW = torch.empty((K, N), dtype=out_dtype, device=dY.device)
    dA = dA if want_dA else None
    dW = dW if want_dW else None
    _check(lib().fp4_linear_backward(_ptr(dY), _dt(dY), M, K, N, _ptr(Aq), _ptr(sA), _ptr(Wq), _ptr(sW), _ptr(dA),
                                     _dt(dA) if dA is not None else FP4_F32, _ptr(dW),
                                     _dt(dW) if dW is not None else FP4_F32, _ptr(ws), ws.numel(), _stream(dY)))
    return dA, dW


def backward_intermediates(ws: torch.Tensor, M: int, K: int, N: int) -> dict:
    """Views of Gq, sG, Hq, sH, WqT and AqT inside a backward workspace."""
    lay = backward_layout(M, K, N)

    def view(off, nbytes, dt, shape):
        return ws[off:off + nbytes].view(dt).view(shape)

    return dict(Gq=view(lay.Gq, M * (N // 2), torch.uint8, (M, N // 2)), sG=view(lay.sG, 4 * M, torch.float32, (M,)),
                Hq=view(lay.Hq, N * (M // 2), torch.uint8, (N, M // 2)), sH=view(lay.sH, 4 * N, torch.float32, (N,)),
                WqT=view(lay.WqT, K * (N // 2), torch.uint8, (K, N // 2)),
                AqT=view(lay.AqT, K * (M // 2), torch.uint8, (K, M // 2)))


# --------------------------------------------------------------------------- FP8 linear layer, blocks of 128
class Block8:
    """An E4M3 operand: `rows` rows of contraction length `length`, one power-of-two scale per
    block of 128 along the contraction (FP4_BLOCK_VECTOR) or per 128 x 128 block (FP4_BLOCK_SQUARE).
    codes: u8 (rows, length rounded up to 128); scales: u8, laid out as the C header says."""
    __slots__ = ("codes", "scales", "rows", "length", "mode")

    def __init__(self, rows: int, length: int, mode: int, device):
        n = lib().fp4_block8_scales_bytes(rows, length, mode)
        if n == 0:
            raise Fp4Error(f"no block-128 operand of {rows} rows, contraction {length}, mode {mode}")
        self.rows, self.length, self.mode = rows, length, mode
        self.codes = torch.empty(rows, (length + 127) // 128 * 128, dtype=torch.uint8, device=device)
        self.scales = torch.empty(n, dtype=torch.uint8, device=device)


def _need_rows(*ts):
    """Matrices on a HIP device whose rows are contiguous (any row stride, any alignment)."""
    for t in ts:
        if t.is_cuda and t.is_contiguous() and t.dim() == 2:
            continue
        if not t.is_cuda or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or \
                (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
            raise ValueError("expected a matrix on a HIP device with contiguous rows")


def _ld(t: torch.Tensor) -> int:
    return max(t.stride(0), t.shape[1])


def _same_device(ref: torch.Tensor, *ts):
    d = ref.get_device()
    for t in ts:
        if t is not None and t.get_device() != d:
            raise ValueError("tensors must be on one device")


def _scratch(ws: torch.Tensor | None, nbytes: int, ref: torch.Tensor) -> torch.Tensor:
    """A given workspace, all of it memory of ref's device, or a new one."""
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=ref.device)
    _need_cuda(ws)
    _same_device(ref, ws)
    return ws


def block8_quantize(X: torch.Tensor, mode: int = FP4_BLOCK_VECTOR, rows: bool = True, cols: bool = False):
    """(operand of X, operand of X transposed), each None when not asked for.  For a weight W (K x N)
    in FP4_BLOCK_SQUARE, cols is the forward's operand and rows the one dX contracts with."""
    _need_rows(X)
    R, Cn = X.shape
    r = Block8(R, Cn, mode, X.device) if rows else None
    c = Block8(Cn, R, mode, X.device) if cols else None
    _check(lib().fp4_block8_quantize(_ptr(X), _dt(X), R, Cn, _ld(X), mode, _ptr(r.codes) if r else None,
                                     _ptr(r.scales) if r else None, _ptr(c.codes) if c else None,
                                     _ptr(c.scales) if c else None, _stream(X)))
    return r, c


def block8_dequantize(op: Block8, out_dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """The values that an operand stands for (rows x length)."""
    Y = torch.empty((op.rows, op.length), dtype=out_dtype, device=op.codes.device)
    _check(lib().fp4_block8_dequantize(_ptr(op.codes), _ptr(op.scales), op.rows, op.length, op.mode, _ptr(Y),
                                       _out_dtype_code(out_dtype), _stream(Y)))
    return Y


def block8_gemm(a: Block8, b: Block8, out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """a . b^T of two operands with one contraction length."""
    if a.length != b.length:
        raise ValueError(f"contraction lengths differ: {a.length} and {b.length}")
    _same_device(a.codes, b.codes)
    Y = torch.empty((a.rows, b.rows), dtype=out_dtype, device=a.codes.device)
    _check(lib().fp4_block8_gemm(_ptr(a.codes), _ptr(a.scales), a.mode, _ptr(b.codes), _ptr(b.scales), b.mode, a.rows,
                                 b.rows, a.length, _ptr(Y), _out_dtype_code(out_dtype), _stream(Y)))
    return Y


def block8_linear_forward(x: torch.Tensor, w: Block8, out_dtype: torch.dtype | None = None, for_backward: bool = False,
                          ws: torch.Tensor | None = None):
    """y = x . W with x (M x K, fp32 or bf16) quantized in blocks of 128 along K and W given by
    block8_quantize(W, FP4_BLOCK_SQUARE, cols=True)[1].  for_backward: (y, operand of x transposed)."""
    _need_rows(x)
    M, K = x.shape
    if K != w.length:
        raise ValueError(f"x has {K} columns, the weight a contraction of {w.length}")
    _same_device(x, w.codes)
    Y = torch.empty(M, w.rows, dtype=out_dtype or x.dtype, device=x.device)
    if M == 0:
        if for_backward:
            raise ValueError("no rows to contract in the backward")
        return Y
    L = lib()
    xt = Block8(K, M, FP4_BLOCK_VECTOR, x.device) if for_backward else None
    ws = _scratch(ws, L.fp4_block8_linear_workspace_bytes(M, K, w.rows), x)
    _check(L.fp4_block8_linear(_ptr(x), _dt(x), M, K, _ld(x), _ptr(w.codes), _ptr(w.scales), w.mode, w.rows, _ptr(Y),
                               _dt(Y), _ptr(xt.codes) if xt else None, _ptr(xt.scales) if xt else None, _ptr(ws),
                               ws.numel(), _stream(x)))
    return (Y, xt) if for_backward else Y


def block8_linear_backward(dy: torch.Tensor, w: Block8 | None, xt: Block8 | None, out_dtype: torch.dtype | None = None,
                           ws: torch.Tensor | None = None):
    """(dx, dw) from dy (M x N), W's operand of K rows (block8_quantize's rows) and the operand of x
    transposed (block8_linear_forward's); w or xt None: that gradient is not wanted (None)."""
    _need_rows(dy)
    if w is None and xt is None:
        raise ValueError("no gradient asked for")
    M, N = dy.shape
    K = w.rows if w is not None else xt.rows
    if (w is not None and w.length != N) or (xt is not None and (xt.length != M or xt.rows != K)):
        raise ValueError("operands do not fit dy")
    if xt is not None and xt.mode != FP4_BLOCK_VECTOR:
        raise ValueError("the activation's operand has vector blocks")
    _same_device(dy, w.codes if w is not None else None, xt.codes if xt is not None else None)
    out_dtype = out_dtype or dy.dtype
    dx = torch.empty(M, K, dtype=out_dtype, device=dy.device) if w is not None else None
    dw = torch.empty(K, N, dtype=out_dtype, device=dy.device) if xt is not None else None
    L = lib()
    ws = _scratch(ws, L.fp4_block8_backward_workspace_bytes(M, N), dy)
    od = _out_dtype_code(out_dtype)
    _check(L.fp4_block8_backward(_ptr(dy), _dt(dy), M, K, N, _ld(dy), _ptr(w.codes) if w is not None else None,
                                 _ptr(w.scales) if w is not None else None, w.mode if w is not None else 0,
                                 _ptr(xt.codes) if xt is not None else None, _ptr(xt.scales) if xt is not None else None,
                                 _ptr(dx), od, _ptr(dw), od, _ptr(ws), ws.numel(), _stream(dy)))
    return dx, dw


# --------------------------------------------------------------------------- 4-bit key/value cache
class KV4Cache:
    """A paged cache of keys and values in 4 bits (data: u8, laid out as the C header's library
    does; pages x page tokens x heads x d)."""
    __slots__ = ("data", "pages", "page", "heads", "d")

    def __init__(self, data, pages, page, heads, d):
        self.data, self.pages, self.page, self.heads, self.d = data, pages, page, heads, d


def kv4_cache(pages: int, page: int, heads: int, d: int, device="cuda") -> KV4Cache:
    """An empty cache: page (tokens) a power of two from 16 to 1024, d 64 or 128."""
    n = lib().fp4_kv4_cache_bytes(pages, page, heads, d)
    if n == 0:
        raise Fp4Error(f"no 4-bit cache of {pages} pages of {page} tokens, {heads} heads of {d}")
    return KV4Cache(torch.zeros(n, dtype=torch.uint8, device=device), pages, page, heads, d)


def _slot_bytes(t: torch.Tensor, n: int) -> int:
    if t.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"expected int32 or int64 indices, got {t.dtype}")
    if not t.is_cuda or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"expected {n} contiguous indices on a HIP device")
    return t.element_size()


def kv4_write(cache: KV4Cache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
    """Quantize k and v (n x heads x d, fp32 or bf16, d contiguous) into the cache at slots (page index *
    page + offset; those outside the cache are skipped, and the others must differ)."""
    n = k.shape[0]
    shape = (n, cache.heads, cache.d)
    for t in (k, v):
        if not t.is_cuda or t.shape != shape or t.stride(2) != 1:
            raise ValueError(f"expected (n, {cache.heads}, {cache.d}) on a HIP device, the last dimension contiguous")
    if k.dtype != v.dtype:
        raise TypeError("k and v must share a dtype")
    sb = _slot_bytes(slots, n)
    _same_device(cache.data, k, v, slots)
    if n == 0:
        return
    _check(lib().fp4_kv4_write(_ptr(cache.data), cache.pages, cache.page, cache.heads, cache.d, _ptr(k), _ptr(v), _dt(k),
                               n, k.stride(0), k.stride(1), v.stride(0), v.stride(1), _ptr(slots), sb, _stream(k)))


def kv4_read(cache: KV4Cache, slots: torch.Tensor, d: int | None = None, out_dtype: torch.dtype = torch.bfloat16):
    """(k, v), n x heads x d, of the tokens at slots; d, if given, must be the cache's."""
    if d is not None and d != cache.d:
        raise ValueError(f"the cache holds heads of {cache.d}")
    n = slots.numel()
    sb = _slot_bytes(slots, n)
    _same_device(cache.data, slots)
    k = torch.empty(n, cache.heads, cache.d, dtype=out_dtype, device=slots.device)
    v = torch.empty_like(k)
    if n:
        _check(lib().fp4_kv4_read(_ptr(cache.data), cache.pages, cache.page, cache.heads, cache.d, _ptr(slots), sb, n,
                                  _ptr(k), _ptr(v), _out_dtype_code(out_dtype), _stream(slots)))
    return k, v


def kv4_attention_workspace(q: torch.Tensor, cache: KV4Cache, pages: torch.Tensor, max_q: int = 1,
                            shared: int = 0) -> torch.Tensor:
    """A workspace for kv4_attention with these sizes and any window and sinks (max_q as there: q's rows if it is not given
    with q_start)."""
    b, width = pages.shape
    if shared and b and q.shape[0]:
        n = lib().fp4_kv4_attention_shared_workspace_bytes(q.shape[0], b, max_q, q.shape[1], cache.heads, cache.d, cache.page,
                                                           width, shared)
    else:
        n = lib().fp4_kv4_attention_workspace_bytes(b, max_q, q.shape[1], cache.heads, cache.d, cache.page, width)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)


def kv4_attention(q: torch.Tensor, cache: KV4Cache, pages: torch.Tensor, lens: torch.Tensor,
                  q_start: torch.Tensor | None = None, max_q: int | None = None, window: int = 0, scale: float | None = None,
                  return_lse: bool = False, ws: torch.Tensor | None = None, sinks: int = 0, shared: int = 0):
    """Causal attention of packed bf16 queries q (nq x hq x d) over the cache.  pages: int32 page table
    (b x width); lens: int32 tokens of each sequence in the cache, its queries' own among them; q_start: int32
    b + 1 offsets of the sequences' queries, or None for one query a sequence; max_q: the most queries of a
    sequence (None: as many as q has, or 1 without q_start; a close bound is faster, needs less workspace, and is
    needed where b times q's rows pass what a call may have);
    window: tokens a query sees (0: all); sinks: with a window, the first tokens of a sequence that stay visible;
    shared: the first pages of every row that are taken to be row 0's, and read once for all sequences where that is
    quicker (not with a window; ws of kv4_attention_workspace with the same shared).  A query that sees nothing gets 0 and lse -inf, and so does one past its
    sequence's first max_q, before q_start[0] or from q_start[b] on."""
    if q.dtype is not torch.bfloat16:
        raise TypeError(f"expected bfloat16 queries, got {q.dtype}")
    # (each attribute of a tensor costs about 0.1 us: they are read once)
    dev, qs, qst, ps, pst = q.get_device(), q.shape, q.stride(), pages.shape, pages.stride()
    if dev < 0 or len(qs) != 3 or qs[2] != cache.d or qst[2] != 1:
        raise ValueError(f"expected queries (nq, hq, {cache.d}) on a HIP device, the last dimension contiguous")
    nq, hq, d = qs
    if hq == 0 or hq % cache.heads:
        raise ValueError(f"{hq} query heads over {cache.heads} key/value heads")
    if pages.dtype is not torch.int32 or pages.get_device() < 0 or len(ps) != 2 or (ps[1] > 1 and pst[1] != 1) or \
            (ps[0] > 1 and pst[0] < ps[1]):
        raise ValueError("expected an int32 page table (b, width) on a HIP device, rows contiguous")
    b, width = ps
    if lens.dtype is not torch.int32 or lens.get_device() < 0 or lens.shape != (b,) or not lens.is_contiguous():
        raise ValueError(f"expected {b} int32 lengths on a HIP device")
    if q_start is None:
        if nq != b:
            raise ValueError(f"{nq} queries for {b} sequences without q_start")
        if max_q is None:
            max_q = 1
    else:
        if q_start.dtype is not torch.int32 or q_start.get_device() < 0 or q_start.shape != (b + 1,) or not q_start.is_contiguous():
            raise ValueError(f"expected {b + 1} int32 offsets on a HIP device")
        if max_q is None:
            max_q = nq
    if sinks < 0 or shared < 0:
        raise ValueError(f"sinks {sinks}, shared {shared}")
    if shared and window:
        raise ValueError("shared pages and a window do not go together")
    _same_device(q, cache.data, pages, lens, q_start, ws)
    if ws is not None and not ws.is_contiguous():
        raise ValueError("expected a contiguous workspace")
    o = torch.empty_like(q, memory_format=torch.contiguous_format)
    lse = torch.empty(nq, hq, dtype=torch.float32, device=q.device) if return_lse else None
    if nq and not b:  # no sequence owns a query
        o.zero_()
        if return_lse:
            lse.fill_(float("-inf"))
    elif nq:
        if ws is None:
            ws = kv4_attention_workspace(q, cache, pages, max_q, shared)
        L, most = lib(), 0x7FFFFFFF
        if shared:
            f, seen = L.fp4_kv4_attention_shared, (shared,)
        elif sinks and window:
            f, seen = L.fp4_kv4_attention_sinks, (min(window, most), min(sinks, most))
        else:
            f, seen = L.fp4_kv4_attention, (min(window, most),)
        _on_device(q, f, q.data_ptr(), qst[0], qst[1], nq, hq, _ptr(q_start), lens.data_ptr(), b, max_q, pages.data_ptr(),
                   max(pst[0], width), width, cache.data.data_ptr(), cache.pages, cache.page, cache.heads, d, *seen,
                   d ** -0.5 if scale is None else float(scale), o.data_ptr(), _ptr(lse), ws.data_ptr(), ws.numel(), _stream(q))
    return (o, lse) if return_lse else o


# --------------------------------------------------------------------------- page tables of the cache
def _on_device(ref: torch.Tensor, call, *args):
    """call(*args), which enqueues on ref's device, with that device current; raises its status."""
    if torch.cuda.is_initialized() and ref.get_device() != torch._C._cuda_getDevice():
        with torch.cuda.device(ref.device):
            status = call(*args)
    else:
        status = call(*args)
    if status:
        _check(status)


def _int32s(name: str, t: torch.Tensor, shape, ref: torch.Tensor | None = None):
    if t.dtype is not torch.int32 or not t.is_cuda or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"expected {name} as {tuple(shape)} contiguous int32 on a HIP device")
    if ref is not None and t.get_device() != ref.get_device():
        raise ValueError("tensors must be on one device")


class KV4Pages:
    """The page tables of b sequences of a cache and its free pages, all int32 on the device: table (b x width, -1
    where there is no page), lens (b, tokens of each), free (pages) and count (1): the first count entries of free
    are the free pages, the last of them the next to be taken.  The tensors are checked once and stay the object's;
    their values may be written at any time."""
    __slots__ = ("_table", "_lens", "_free", "_count", "_page", "_slots", "_args")

    def __init__(self, table, lens, free, count, page):
        if table.dim() != 2 or free.dim() != 1 or not table.numel() or not free.numel():
            raise ValueError("expected a table (b, width) and a stack of free pages")
        (b, width), pages = table.shape, free.shape[0]
        _int32s("the table", table, (b, width))
        _int32s("the lengths", lens, (b,), table)
        _int32s("the free pages", free, (pages,), table)
        _int32s("their count", count, (1,), table)
        self._table, self._lens, self._free, self._count, self._page = table, lens, free, count, page
        self._slots = torch.empty(0, dtype=torch.int64, device=table.device)
        self._args = (_ptr(table), width, b, width, _ptr(lens), _ptr(free), _ptr(count), pages, page)

    table = property(lambda self: self._table)
    lens = property(lambda self: self._lens)
    free = property(lambda self: self._free)
    count = property(lambda self: self._count)
    pages = property(lambda self: self._args[7])
    page = property(lambda self: self._page)


def kv4_page_tables(b: int, width: int, pages: int, page: int, device="cuda") -> KV4Pages:
    """Empty tables of b sequences, up to width pages each, over a cache of `pages` pages of `page` tokens, all free
    (page 0 is taken first)."""
    if b < 1 or width < 1 or not 1 <= pages <= 0x7FFFFFFF or page < 16 or page > 1024 or page & (page - 1):
        raise Fp4Error(f"no page tables of {b} sequences of {width} pages over {pages} pages of {page} tokens")
    i32 = dict(dtype=torch.int32, device=device)
    return KV4Pages(torch.full((b, width), -1, **i32), torch.zeros(b, **i32), torch.arange(pages - 1, -1, -1, **i32),
                    torch.full((1,), pages, **i32), page)


def kv4_extend(tables: KV4Pages, new: torch.Tensor | None = None, n: int | None = None):
    """Append new[i] tokens (int32, b; None: one each) to sequence i: takes pages, writes the table, adds to the lengths.
    With n, the call's tokens lie one sequence after the other: (slots, positions, q_start), slots int64 and positions
    int32 for n tokens (-1 behind the last), q_start int32 b + 1; q_start[i+1] - q_start[i] is what sequence i got:
    new[i], or 0 where its row, the free pages or n did not suffice.  Without n, token i is sequence i's only one:
    (slots, positions), -1 where it got none (new[i] = 0: none; above 1 counts as 1)."""
    lens = tables._lens
    b = lens.shape[0]
    if new is not None:
        _int32s("the new tokens", new, (b,), lens)
    elif n is not None:
        raise ValueError("n tokens need new")
    L = lib()
    if n is None:
        m, q_start, need, ws = b, None, 0, None
    else:
        if n < 0:
            raise ValueError(f"{n} tokens")
        m, q_start = n, lens.new_empty(b + 1)
        need = L.fp4_kv4_extend_workspace_bytes(b, n)
        ws = lens.new_empty(need // 4) if need else None
    slots, pos = tables._slots.new_empty(m), lens.new_empty(m)
    _on_device(lens, L.fp4_kv4_extend, *tables._args, _ptr(new), m, slots.data_ptr(), pos.data_ptr(), _ptr(q_start), _ptr(ws),
               need, _stream(lens))
    return (slots, pos) if n is None else (slots, pos, q_start)


def kv4_release(tables: KV4Pages, keep: torch.Tensor | None = None, window: int = 0, sinks: int = 0, shared: int = 0) -> None:
    """Cut sequence i to its first keep[i] tokens (int32, b; None: all stay; 0 ends it) and give back the pages past them,
    and with a window those that no later query sees through it beside the first `sinks` tokens.  The first
    `shared` columns stay.  What is given back first is taken first by the next kv4_extend."""
    lens = tables._lens
    if keep is not None:
        _int32s("the lengths to keep", keep, lens.shape, lens)
    L, most = lib(), 0x7FFFFFFF
    need = L.fp4_kv4_release_workspace_bytes(*tables._args[2:4])
    ws = lens.new_empty(need // 4) if need else None
    _on_device(lens, L.fp4_kv4_release, *tables._args, _ptr(keep), min(window, most), min(sinks, most), min(shared, most),
               _ptr(ws), need, _stream(lens))


# --------------------------------------------------------------------------- norm of queries and keys, rotation
def rope_table(max_pos: int, rot: int, base: float = 10000.0, factor: float = 1.0, device="cuda") -> torch.Tensor:
    """fp32 (max_pos, rot): the rot / 2 cosines, then the rot / 2 sines, of pos / factor * base^(-2 i / rot)."""
    t = torch.empty(max_pos, rot, dtype=torch.float32, device=device)
    if not t.is_cuda:
        raise ValueError("expected a HIP device")
    _on_device(t, lib().fp4_rope_table, _ptr(t), max_pos, rot, float(base), float(factor), _stream(t))
    return t


def _head_args(name: str, t: torch.Tensor, dtype: torch.dtype, dev: int, n: int, d: int):
    """C arguments (pointer, token and head strides) of t as n x heads x d on device dev, and the heads."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[0] != n or shape[2] != d or stride[2] != 1:
        raise ValueError(f"expected {name} as ({n}, heads, {d}), the last dimension contiguous")
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if t.get_device() != dev:
        raise ValueError("tensors must be on one device")
    return (t.data_ptr(), stride[0], stride[1]), shape[1]


_NO_HEADS = ((None, 0, 0), 0)


def _weight_args(w: torch.Tensor, dev: int, d: int) -> int:
    """w's type code, after its checks."""
    if w.get_device() != dev or w.dim() != 1 or w.numel() != d or not w.is_contiguous():
        raise ValueError(f"expected {d} contiguous weights on the rows' device")
    return _dt(w)


def _rope_args(q, k, table, positions, q_weight, k_weight, eps):
    """Checks what the calls over rows of heads share: (n, d, device, q's and k's arguments, those from the weights to rot)."""
    dev, dtype = q.get_device(), q.dtype
    if dev < 0 or q.dim() != 3:
        raise ValueError("expected queries (n, heads, d) on a HIP device")
    n, _, d = q.shape
    qa = _head_args("q", q, dtype, dev, n, d)
    ka = _NO_HEADS if k is None else _head_args("k", k, dtype, dev, n, d)
    if qa[1] == 0:
        raise ValueError("no query heads")
    wdt = FP4_F32
    if q_weight is not None or k_weight is not None:
        if eps is None:
            raise ValueError("weights without a norm")
        if k is None and k_weight is not None:
            raise ValueError("weights without keys")
        wdt = _weight_args(q_weight if q_weight is not None else k_weight, dev, d)
        if q_weight is not None and k_weight is not None and _weight_args(k_weight, dev, d) != wdt:
            raise TypeError("the weights must share a dtype")
    if eps is not None and not eps >= 0:
        raise ValueError(f"eps {eps}")
    if table is None:
        pos = tab = None
        max_pos = rot = 0
    else:
        if table.dtype is not torch.float32 or table.get_device() != dev or table.dim() != 2 or not table.is_contiguous():
            raise ValueError("expected an fp32 table (max_pos, rot) on the rows' device")
        if positions is None:
            raise ValueError("a table without positions")
        if positions.dtype is not torch.int32 or positions.get_device() != dev or positions.dim() != 1 or \
                positions.numel() != n or not positions.is_contiguous():
            raise ValueError(f"expected {n} contiguous int32 positions on the rows' device")
        max_pos, rot = table.shape
        if rot < 16:
            raise ValueError(f"a rotation of {rot} columns")
        pos, tab = positions.data_ptr(), table.data_ptr()
    return n, d, dev, qa, ka, (_ptr(q_weight), _ptr(k_weight), wdt, -1.0 if eps is None else float(eps), pos, tab, max_pos, rot)


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None, table: torch.Tensor | None = None,
                 positions: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float | None = 1e-6, interleaved: bool = False):
    """Norm of each head of q (n x hq x d, fp32 or bf16) and k (n x hkv x d, or None), times a weight (d, None: ones), and
    rotation of the first columns by table (rope_table's) at positions (int32, n): dense (q, k).  eps None: no norm; table
    None: no rotation.  Pairs are (i, i + rot / 2), or (2 i, 2 i + 1) if interleaved.  A negative position's rows
    are zeros; one past the table makes the rotated columns NaN."""
    n, d, dev, (qp, hq), (kp, hkv), args = _rope_args(q, k, table, positions, q_weight, k_weight, eps)
    qo = torch.empty_like(q, memory_format=torch.contiguous_format)
    ko = None if k is None else torch.empty_like(k, memory_format=torch.contiguous_format)
    if n:
        _on_device(q, lib().fp4_qk_norm_rope, *qp, hq, *kp, hkv, n, d, _dt(q), *args, int(interleaved), qo.data_ptr(), _ptr(ko),
                   _stream(q))
    return qo, ko


def qk_norm_rope_backward(dq: torch.Tensor, dk: torch.Tensor | None, q: torch.Tensor, k: torch.Tensor | None,
                          table: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                          q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                          eps: float | None = 1e-6, interleaved: bool = False, out=None):
    """Gradients (of q, of k, of q_weight, of k_weight) of qk_norm_rope from those of its outputs and its inputs; the weights'
    in fp32 (None where there is no weight).  out: (tensor or None, tensor or None) for the first two, views into the
    fused projection's gradient for one."""
    n, d, dev, (qp, hq), (kp, hkv), args = _rope_args(q, k, table, positions, q_weight, k_weight, eps)
    if (dk is None) != (k is None):
        raise ValueError("keys and their gradient go together")
    gq, gk = out if out is not None else (None, None)
    if gq is None:
        gq = torch.empty_like(q, memory_format=torch.contiguous_format)
    if gk is None and k is not None:
        gk = torch.empty_like(k, memory_format=torch.contiguous_format)
    elif k is None and gk is not None:
        raise ValueError("a place for a gradient without keys")
    dt = q.dtype
    (dqp, h0), (gqp, h1) = _head_args("dq", dq, dt, dev, n, d), _head_args("out", gq, dt, dev, n, d)
    (dkp, h2), (gkp, h3) = (_NO_HEADS, _NO_HEADS) if k is None else (_head_args("dk", dk, dt, dev, n, d),
                                                                     _head_args("out", gk, dt, dev, n, d))
    if h0 != hq or h1 != hq or h2 != hkv or h3 != hkv:
        raise ValueError("gradients are not like the inputs")
    wq = wk = ws = None
    need = 0
    if q_weight is not None or k_weight is not None:
        wq, wk = torch.empty(2, d, dtype=torch.float32, device=q.device).unbind(0)
        wq, wk = wq if q_weight is not None else None, wk if k_weight is not None else None
        need = lib().fp4_qk_norm_rope_backward_workspace_bytes(d)
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    if n:
        _on_device(q, lib().fp4_qk_norm_rope_backward, *dqp, *dkp, *qp, hq, *kp, hkv, n, d, _dt(q), *args, int(interleaved), *gqp,
                   *gkp, _ptr(wq), _ptr(wk), _ptr(ws), need, _stream(q))
    else:
        for w in (wq, wk):
            if w is not None:
                w.zero_()
    return gq, gk, wq, wk


def kv4_norm_rope(cache: KV4Cache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                  table: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                  q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float | None = 1e-6,
                  interleaved: bool = False) -> torch.Tensor:
    """qk_norm_rope, of which k goes with v (n x heads x d) to the cache's slots (as kv4_write takes them) in the same
    launch: returns q."""
    n, d, dev, (qp, hq), (kp, hkv), args = _rope_args(q, k, table, positions, q_weight, k_weight, eps)
    vp, hv = _head_args("v", v, q.dtype, dev, n, d)
    if hkv != cache.heads or hv != hkv or d != cache.d:
        raise ValueError(f"expected keys and values (n, {cache.heads}, {cache.d})")
    sb = _slot_bytes(slots, n)
    _same_device(q, cache.data, slots)
    qo = torch.empty_like(q, memory_format=torch.contiguous_format)
    if n:
        _on_device(q, lib().fp4_kv4_norm_rope, cache.data.data_ptr(), cache.pages, cache.page, *qp, hq, *kp, *vp, hkv, n, d,
                   _dt(q), slots.data_ptr(), sb, *args, int(interleaved), qo.data_ptr(), _stream(q))
    return qo
