"""Row-wise-scaled FP8 linear layer with a 2:4 sparse weight, for MI355X (gfx950).

Thin Python binding of ``libsparse_fp8_row.so`` (C ABI in
``include/sparse_fp8_row.h``).  This module only marshals arguments: every
step of the computation runs in the library's HIP kernels.  PyTorch provides
device memory and the current HIP stream.

    xq, xs = quantize_rowwise_fp8(x)                    # x: bf16 [M, K] on the GPU
    w = prepare_weight(w_bf16, torch.float8_e4m3fn)     # once per weight
    y = sparse_fp8_rowwise_linear(xq, xs, w.values, w.meta, w.scale, bias)

Tensor-wise scaling (one scale per operand): ``quantize_tensorwise_fp8``,
``prepare_weight(..., scaling="tensor")`` and ``sparse_fp8_scaled_linear``.

The gated feed-forward block (``gated_linear``, its gradients from 8-bit
activations, its 4-bit form) and the MX block formats, the linear layer in
8-bit integers (``int8_linear``) and the mixture of gated blocks for a few
tokens (``moe_route``, ``moe_layer``) are at the end of this module.  None of
these calls builds an autograd graph: the gated block's gradient is
``gated_linear_backward``.

The operator follows pytorch/ao PR #1671 ("Add CUTLASS-based row-wise scaled
sparse FP8 kernel"); see the header for the exact contract of each call.
There is no fallback: if the library is missing or no GPU is present the
calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsparse_fp8_row.so")

SFR_E4M3, SFR_E5M2 = 0, 1
SFR_OUT_BF16, SFR_OUT_F32 = 0, 1
SFR_SCALE_ROW, SFR_SCALE_TENSOR = 0, 1
STATUS = {0: "SFR_OK", 1: "SFR_ERR_NULL", 2: "SFR_ERR_SHAPE", 3: "SFR_ERR_ALIGN",
          4: "SFR_ERR_DTYPE", 5: "SFR_ERR_LAUNCH"}
EXPORTED = ("quantize_rowwise_fp8", "quantize_tensorwise_fp8", "sfr_quantize_tensorwise_workspace_bytes",
            "quantize_tensorwise_fp8_noalloc",
            "compress_2to4_fp8", "prune_2to4_bf16", "sparse_fp8_rowwise_linear", "sparse_fp8_scaled_linear",
            "sparse_fp8_rowwise_linear_dynamic", "sparse_fp8_rowwise_linear_dynamic_algo",
            "sparse_fp8_scaled_linear_algo", "sfr_linear_algo_count", "sfr_linear_algo_valid",
            "sfr_linear_algo_name", "sfr_linear_algo_supported", "sfr_linear_default_algo",
            "bsr_count_bf16", "bsr_fill_bf16", "bsr_linear_bf16", "sfr_status_string", "sfr_format_version",
            "quantize_mx", "dequantize_mx", "gated_linear_bf16", "gated_linear_bf16_backward",
            "sfr_gated_backward_workspace_bytes", "mxfp4_linear", "mxfp4_gated_linear", "sfr_mxfp4_workspace_bytes",
            "sfr_block_kernel",
            "quantize_rowwise_int8", "int8_scaled_linear", "int8_linear_dynamic", "sfr_int8_workspace_bytes",
            "sfr_int8_kernel", "moe_route", "moe_layer", "sfr_moe_workspace_bytes")

_FP8 = {torch.float8_e4m3fn: SFR_E4M3, torch.float8_e5m2: SFR_E5M2}
_lib = None


class SfrError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}")
        self.status = status


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the HIP library (torch is imported first so both share one HIP runtime)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run `python -m sparse_fp8_row_amd.build`")
    lib = ctypes.CDLL(path)
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.quantize_rowwise_fp8.argtypes = [P, I64, I64, I, P, P, P]
    lib.compress_2to4_fp8.argtypes = [P, I64, I64, I, P, P, P]
    lib.prune_2to4_bf16.argtypes = [P, I64, I64, P, P]
    lib.sparse_fp8_rowwise_linear.argtypes = [P, I, P, I64, I64, P, P, I, P, I64, P, P, I, P]
    lib.quantize_tensorwise_fp8.argtypes = [P, I64, I64, I, P, P, P, I64, P]
    lib.quantize_tensorwise_fp8_noalloc.argtypes = [P, I64, I64, I, P, P, P]
    lib.quantize_tensorwise_fp8_noalloc.restype = I
    lib.sparse_fp8_scaled_linear.argtypes = [P, I, P, I, I64, I64, P, P, I, P, I, I64, P, P, I, P]
    lib.sparse_fp8_rowwise_linear_dynamic.argtypes = [P, I, I64, I64, P, P, I, P, I, I64, P, P, I, P, P, P]
    lib.sparse_fp8_rowwise_linear_dynamic_algo.argtypes = [P, I, I64, I64, P, P, I, P, I, I64, P, P, I, P, P, I, P]
    lib.sfr_linear_algo_valid.argtypes = [I]
    lib.sfr_linear_algo_valid.restype = I
    lib.sparse_fp8_scaled_linear_algo.argtypes = [P, I, P, I, I64, I64, P, P, I, P, I, I64, P, P, I, I, P]
    lib.sparse_fp8_scaled_linear_algo.restype = I
    lib.sfr_linear_algo_count.argtypes = []
    lib.sfr_linear_algo_count.restype = I
    lib.sfr_linear_algo_name.argtypes = [I]
    lib.sfr_linear_algo_name.restype = ctypes.c_char_p
    lib.sfr_linear_algo_supported.argtypes = [I, I64, I64, I64]
    lib.sfr_linear_algo_supported.restype = I
    lib.sfr_linear_default_algo.argtypes = [I64, I64, I64]
    lib.sfr_linear_default_algo.restype = I
    lib.bsr_count_bf16.argtypes = [P, I64, I64, P, P]
    lib.bsr_fill_bf16.argtypes = [P, I64, I64, P, P, P, P]
    lib.bsr_linear_bf16.argtypes = [P, I64, I64, P, P, P, I64, P, P, I, P]
    lib.quantize_mx.argtypes = [P, I64, I64, I, P, P, P]
    lib.dequantize_mx.argtypes = [P, P, I64, I64, I, P, P]
    lib.gated_linear_bf16.argtypes = [P, I64, I64, P, I64, I, P, I, P, P, P]
    lib.gated_linear_bf16_backward.argtypes = [P, I64, I64, I64, I, P, P, I, P, P, I, P, P, P, P, I64, P]
    lib.mxfp4_linear.argtypes = [P, I64, I64, P, P, I64, P, P, I, P, I64, P]
    lib.mxfp4_gated_linear.argtypes = [P, I64, I64, P, P, I64, I, P, P]
    lib.sfr_gated_backward_workspace_bytes.argtypes = [I64, I64, I64, I]
    lib.sfr_gated_backward_workspace_bytes.restype = I64
    lib.sfr_mxfp4_workspace_bytes.argtypes = [I64, I64, I64]
    lib.sfr_mxfp4_workspace_bytes.restype = I64
    lib.sfr_block_kernel.argtypes = [I, I64, I64, I64, ctypes.POINTER(ctypes.c_int32)]
    lib.sfr_block_kernel.restype = ctypes.c_char_p
    lib.quantize_rowwise_int8.argtypes = [P, I64, I64, P, P, P]
    lib.int8_scaled_linear.argtypes = [P, P, I64, I64, P, P, I64, P, P, I, P, I64, P]
    lib.int8_linear_dynamic.argtypes = [P, I64, I64, P, P, I64, P, P, I, P, I64, P]
    lib.sfr_int8_workspace_bytes.argtypes = [I64, I64, I64, I]
    lib.sfr_int8_workspace_bytes.restype = I64
    lib.sfr_int8_kernel.argtypes = [I64, I64, I64, I, ctypes.POINTER(ctypes.c_int32)]
    lib.sfr_int8_kernel.restype = ctypes.c_char_p
    lib.moe_route.argtypes = [P, I64, I64, P, I64, P, I64, I, I, P, P, P, P]
    lib.moe_layer.argtypes = [P, I64, I64, P, P, I64, I64, I64, I, P, P, P, P, I, P, P, I64, P]
    lib.sfr_moe_workspace_bytes.argtypes = [I64, I64, I64, I64]
    lib.sfr_moe_workspace_bytes.restype = I64
    for fn in (lib.quantize_rowwise_int8, lib.int8_scaled_linear, lib.int8_linear_dynamic, lib.moe_route,
               lib.moe_layer):
        fn.restype = I
    for fn in (lib.quantize_mx, lib.dequantize_mx, lib.gated_linear_bf16, lib.gated_linear_bf16_backward,
               lib.mxfp4_linear, lib.mxfp4_gated_linear):
        fn.restype = I
    for fn in (lib.quantize_rowwise_fp8, lib.compress_2to4_fp8, lib.prune_2to4_bf16, lib.sparse_fp8_rowwise_linear,
               lib.quantize_tensorwise_fp8, lib.sparse_fp8_scaled_linear, lib.sparse_fp8_rowwise_linear_dynamic,
               lib.sparse_fp8_rowwise_linear_dynamic_algo,
               lib.bsr_count_bf16, lib.bsr_fill_bf16, lib.bsr_linear_bf16):
        fn.restype = I
    lib.sfr_quantize_tensorwise_workspace_bytes.argtypes = [I64, I64]
    lib.sfr_quantize_tensorwise_workspace_bytes.restype = I64
    lib.sfr_status_string.argtypes = [I]
    lib.sfr_status_string.restype = ctypes.c_char_p
    lib.sfr_format_version.argtypes = []
    lib.sfr_format_version.restype = I
    if path == LIB_PATH:
        _lib = lib
    return lib


def _check(status: int, where: str):
    if status != 0:
        raise SfrError(status, where)


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _dev(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _fp8_enum(dtype) -> int:
    if dtype not in _FP8:
        raise ValueError(f"unsupported FP8 dtype {dtype}")
    return _FP8[dtype]


def quantize_rowwise_fp8(x: torch.Tensor, dtype=torch.float8_e4m3fn, stream=None):
    """bf16 [rows, cols] -> (q FP8 [rows, cols], scale float32 [rows])."""
    _dev(x, "x")
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    rows, cols = x.shape
    q = torch.empty((rows, cols), dtype=dtype, device=x.device)
    s = torch.empty((rows,), dtype=torch.float32, device=x.device)
    _check(load().quantize_rowwise_fp8(x.data_ptr(), rows, cols, _fp8_enum(dtype), q.data_ptr(),
                                       s.data_ptr(), _stream(stream)), "quantize_rowwise_fp8")
    return q, s


def quantize_tensorwise_fp8(x: torch.Tensor, dtype=torch.float8_e4m3fn, stream=None):
    """bf16 [rows, cols] -> (q FP8 [rows, cols], scale float32 [1]): one scale for the tensor."""
    _dev(x, "x")
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    rows, cols = x.shape
    lib = load()
    q = torch.empty((rows, cols), dtype=dtype, device=x.device)
    s = torch.empty((1,), dtype=torch.float32, device=x.device)
    nbytes = max(int(lib.sfr_quantize_tensorwise_workspace_bytes(rows, cols)), 16)
    work = torch.empty((nbytes,), dtype=torch.uint8, device=x.device)
    _check(lib.quantize_tensorwise_fp8(x.data_ptr(), rows, cols, _fp8_enum(dtype), q.data_ptr(), s.data_ptr(),
                                       work.data_ptr(), nbytes, _stream(stream)), "quantize_tensorwise_fp8")
    return q, s


def quantize_tensorwise_fp8_noalloc(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, stream=None):
    """quantize_tensorwise_fp8 into caller-provided q FP8 [rows, cols] and
    scale float32 [1], on the library's own device workspace (the call
    allocates nothing).  Calls that overlap on one GPU must be serialized."""
    for t, nm in ((x, "x"), (q, "q"), (scale, "scale")):
        _dev(t, nm)
    if x.dtype != torch.bfloat16 or x.dim() != 2 or q.shape != x.shape or scale.shape != (1,) or \
            scale.dtype != torch.float32:
        raise ValueError("x bf16 [rows, cols], q FP8 [rows, cols], scale float32 [1]")
    rows, cols = x.shape
    _check(load().quantize_tensorwise_fp8_noalloc(x.data_ptr(), rows, cols, _fp8_enum(q.dtype), q.data_ptr(),
                                                  scale.data_ptr(), _stream(stream)),
           "quantize_tensorwise_fp8_noalloc")
    return q, scale


def compress_2to4_fp8(wq: torch.Tensor, stream=None):
    """FP8 [n, k] -> (values FP8 [n, k/2], meta uint8 [n, k/8])."""
    _dev(wq, "wq")
    n, k = wq.shape
    values = torch.empty((n, k // 2), dtype=wq.dtype, device=wq.device)
    meta = torch.empty((n, k // 8), dtype=torch.uint8, device=wq.device)
    _check(load().compress_2to4_fp8(wq.data_ptr(), n, k, _fp8_enum(wq.dtype), values.data_ptr(),
                                    meta.data_ptr(), _stream(stream)), "compress_2to4_fp8")
    return values, meta


def prune_2to4_bf16(w: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """bf16 [n, k] -> the same with each group of four along k pruned to its
    two largest magnitudes (the others +0.0).  out may be w (in place)."""
    _dev(w, "w")
    if w.dtype != torch.bfloat16 or w.dim() != 2:
        raise ValueError("w must be a 2-D bfloat16 tensor")
    n, k = w.shape
    if out is None:
        out = torch.empty_like(w)
    elif out.shape != w.shape or out.dtype != w.dtype or not out.is_contiguous():
        raise ValueError("out has the wrong shape or dtype")
    _check(load().prune_2to4_bf16(w.data_ptr(), n, k, out.data_ptr(), _stream(stream)), "prune_2to4_bf16")
    return out


SFR_ALGO_DEFAULT = -1
# Flag of an algorithm id: FP8 matrix-instruction accumulation (twice the
# instruction rate; the products of one 128-k step are added 13 bits below
# the largest).  Without it the accumulation is binary32-grade.
SFR_ALGO_ACC_F8 = 0x100
# Algorithm table consulted by sparse_fp8_scaled_linear when no algo is given:
# {(m_bucket, n, k): algo}, filled by set_algo_table (see tune.py).
_algo_table = {}
M_BUCKETS = (1, 4, 16, 64, 256, 1024, 4096, 1 << 62)


def m_bucket(m: int) -> int:
    """Upper bound of m's bucket: rows 1, 2-4, 5-16, 17-64, ... share a table entry."""
    for b in M_BUCKETS:
        if m <= b:
            return b
    return M_BUCKETS[-1]


def linear_algos(acc: Optional[str] = None):
    """[(id, name)] of the linear layer's algorithms: every kernel
    configuration with binary32-grade accumulation (acc="f32"), with FP8
    matrix-instruction accumulation (acc="f8"), or both (None)."""
    lib = load()
    flags = {"f32": (0,), "f8": (SFR_ALGO_ACC_F8,), None: (0, SFR_ALGO_ACC_F8)}[acc]
    ids = [i | f for f in flags for i in range(lib.sfr_linear_algo_count())]
    return [(a, lib.sfr_linear_algo_name(a).decode()) for a in ids if lib.sfr_linear_algo_valid(a)]


def algo_acc(algo: int) -> str:
    """Accumulation of an algorithm id: "f8" or "f32"."""
    return "f8" if algo >= 0 and algo & SFR_ALGO_ACC_F8 else "f32"


def algo_supported(algo: int, m: int, n: int, k: int) -> bool:
    return bool(load().sfr_linear_algo_supported(algo, m, n, k))


def default_algo(m: int, n: int, k: int) -> int:
    return int(load().sfr_linear_default_algo(m, n, k))


def set_algo_table(table: dict):
    """Use {(m_bucket, n, k): algo} (e.g. from tune.search) for later calls; an
    entry whose algorithm cannot run a shape is ignored for that shape."""
    _algo_table.clear()
    _algo_table.update({(int(b), int(n), int(k)): int(a) for (b, n, k), a in table.items()})


def _table_algo(m: int, n: int, k: int) -> int:
    a = _algo_table.get((m_bucket(m), n, k), SFR_ALGO_DEFAULT)
    return a if a == SFR_ALGO_DEFAULT or algo_supported(a, m, n, k) else SFR_ALGO_DEFAULT


def sparse_fp8_scaled_linear(xq: torch.Tensor, xs: torch.Tensor, values: torch.Tensor, meta: torch.Tensor,
                             ws: torch.Tensor, bias: Optional[torch.Tensor] = None,
                             out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None, stream=None,
                             algo: Optional[int] = None):
    """out[m, n] = xs * ws * sum_k xq[m, k] * wq[n, k] (+ bias[n]), as bf16 (or float32).

    Each scale is per row (xs [m], ws [n]) or one for the tensor (shape [1]);
    the granularity follows from the scale's length.  `algo` picks the kernel
    configuration (see linear_algos); None uses the table set by
    set_algo_table, else the library's built-in choice."""
    for t, nm in ((xq, "xq"), (xs, "xs"), (values, "values"), (meta, "meta"), (ws, "ws")):
        _dev(t, nm)
    m, k = xq.shape
    n = values.shape[0]
    if values.shape != (n, k // 2) or meta.shape != (n, k // 8):
        raise ValueError("operand shapes do not match")
    if xs.dim() != 1 or ws.dim() != 1 or xs.dtype != torch.float32 or ws.dtype != torch.float32:
        raise ValueError("scales must be 1-D float32")
    xk = SFR_SCALE_ROW if xs.shape[0] == m and m != 1 else SFR_SCALE_TENSOR if xs.shape[0] == 1 else None
    wk = SFR_SCALE_ROW if ws.shape[0] == n and n != 1 else SFR_SCALE_TENSOR if ws.shape[0] == 1 else None
    if xk is None or wk is None:
        raise ValueError("scales must have one entry per row or a single entry")
    if bias is not None:
        _dev(bias, "bias")
        if bias.dtype != torch.bfloat16 or bias.shape != (n,):
            raise ValueError("bias must be bfloat16 [n]")
    od = {torch.bfloat16: SFR_OUT_BF16, torch.float32: SFR_OUT_F32}[out_dtype]
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=xq.device)
    elif out.shape != (m, n) or out.dtype != out_dtype or not out.is_contiguous():
        raise ValueError("out has the wrong shape or dtype")
    if algo is None:
        algo = _table_algo(m, n, k)
    _check(load().sparse_fp8_scaled_linear_algo(
        xq.data_ptr(), _fp8_enum(xq.dtype), xs.data_ptr(), xk, m, k, values.data_ptr(), meta.data_ptr(),
        _fp8_enum(values.dtype), ws.data_ptr(), wk, n, 0 if bias is None else bias.data_ptr(), out.data_ptr(), od,
        int(algo), _stream(stream)), "sparse_fp8_scaled_linear")
    return out


def sparse_fp8_rowwise_linear(xq: torch.Tensor, xs: torch.Tensor, values: torch.Tensor, meta: torch.Tensor,
                              ws: torch.Tensor, bias: Optional[torch.Tensor] = None,
                              out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None, stream=None):
    """out[m, n] = xs[m] * ws[n] * sum_k xq[m, k] * wq[n, k] (+ bias[n]), as bf16 (or float32)."""
    for t, nm in ((xq, "xq"), (xs, "xs"), (values, "values"), (meta, "meta"), (ws, "ws")):
        _dev(t, nm)
    m, k = xq.shape
    n = values.shape[0]
    if values.shape != (n, k // 2) or meta.shape != (n, k // 8) or xs.shape != (m,) or ws.shape != (n,):
        raise ValueError("operand shapes do not match")
    if xs.dtype != torch.float32 or ws.dtype != torch.float32:
        raise ValueError("scales must be float32")
    if bias is not None:
        _dev(bias, "bias")
        if bias.dtype != torch.bfloat16 or bias.shape != (n,):
            raise ValueError("bias must be bfloat16 [n]")
    od = {torch.bfloat16: SFR_OUT_BF16, torch.float32: SFR_OUT_F32}[out_dtype]
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=xq.device)
    elif out.shape != (m, n) or out.dtype != out_dtype or not out.is_contiguous():
        raise ValueError("out has the wrong shape or dtype")
    _check(load().sparse_fp8_rowwise_linear(
        xq.data_ptr(), _fp8_enum(xq.dtype), xs.data_ptr(), m, k, values.data_ptr(), meta.data_ptr(),
        _fp8_enum(values.dtype), ws.data_ptr(), n, 0 if bias is None else bias.data_ptr(), out.data_ptr(), od,
        _stream(stream)), "sparse_fp8_rowwise_linear")
    return out


def sparse_fp8_rowwise_linear_dynamic(x: torch.Tensor, values: torch.Tensor, meta: torch.Tensor, ws: torch.Tensor,
                                      bias: Optional[torch.Tensor] = None, act_dtype=torch.float8_e4m3fn,
                                      out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None, stream=None,
                                      algo: Optional[int] = None):
    """bf16 x [m, k] -> (out [m, n], xq [m, k], xs [m]): row-wise activation
    quantization and the linear layer, fused into one launch for small decode shapes."""
    for t, nm in ((x, "x"), (values, "values"), (meta, "meta"), (ws, "ws")):
        _dev(t, nm)
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    m, k = x.shape
    n = values.shape[0]
    if values.shape != (n, k // 2) or meta.shape != (n, k // 8) or ws.dim() != 1:
        raise ValueError("operand shapes do not match")
    wk = SFR_SCALE_ROW if ws.shape[0] == n and n != 1 else SFR_SCALE_TENSOR if ws.shape[0] == 1 else None
    if wk is None or ws.dtype != torch.float32:
        raise ValueError("ws must be float32 [n] or [1]")
    if bias is not None:
        _dev(bias, "bias")
        if bias.dtype != torch.bfloat16 or bias.shape != (n,):
            raise ValueError("bias must be bfloat16 [n]")
    od = {torch.bfloat16: SFR_OUT_BF16, torch.float32: SFR_OUT_F32}[out_dtype]
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=x.device)
    elif out.shape != (m, n) or out.dtype != out_dtype or not out.is_contiguous():
        raise ValueError("out has the wrong shape or dtype")
    xq = torch.empty((m, k), dtype=act_dtype, device=x.device)
    xs = torch.empty((m,), dtype=torch.float32, device=x.device)
    _check(load().sparse_fp8_rowwise_linear_dynamic_algo(
        x.data_ptr(), _fp8_enum(act_dtype), m, k, values.data_ptr(), meta.data_ptr(), _fp8_enum(values.dtype),
        ws.data_ptr(), wk, n, 0 if bias is None else bias.data_ptr(), out.data_ptr(), od, xq.data_ptr(),
        xs.data_ptr(), SFR_ALGO_DEFAULT if algo is None else int(algo), _stream(stream)),
        "sparse_fp8_rowwise_linear_dynamic")
    return out, xq, xs


@dataclass
class SparseFp8Weight:
    """A prepared weight: 2:4-compressed FP8 values, metadata and row scales."""
    values: torch.Tensor   # FP8 [N, K/2]
    meta: torch.Tensor     # uint8 [N, K/8]
    scale: torch.Tensor    # float32 [N]
    format_version: int = 1


def prepare_weight(w: torch.Tensor, dtype=torch.float8_e4m3fn, stream=None, scaling: str = "row") -> SparseFp8Weight:
    """bf16 weight [N, K] -> 2:4 magnitude pruning in bf16, FP8 quantization
    (row-wise, or tensor-wise with scaling="tensor"), 2:4 compression.

    The compressor then keeps each group's two survivors; the row scales are
    those of the dense weight, since a row's largest element always survives."""
    if scaling not in ("row", "tensor"):
        raise ValueError("scaling must be 'row' or 'tensor'")
    pruned = prune_2to4_bf16(w, stream=stream)
    if scaling == "row":
        wq, ws = quantize_rowwise_fp8(pruned, dtype, stream)
    else:
        wq, ws = quantize_tensorwise_fp8(pruned, dtype, stream)
    del pruned
    values, meta = compress_2to4_fp8(wq, stream)
    return SparseFp8Weight(values, meta, ws, int(load().sfr_format_version()))


def linear(x: torch.Tensor, w: SparseFp8Weight, bias: Optional[torch.Tensor] = None,
           act_dtype=torch.float8_e4m3fn, stream=None, act_scaling: str = "row") -> torch.Tensor:
    """bf16 x [M, K] -> bf16 [M, N]: dynamic activation quantization (row- or
    tensor-wise) + sparse FP8 GEMM."""
    if act_scaling == "row":
        xq, xs = quantize_rowwise_fp8(x, act_dtype, stream)
    elif act_scaling == "tensor":
        xq, xs = quantize_tensorwise_fp8(x, act_dtype, stream)
    else:
        raise ValueError("act_scaling must be 'row' or 'tensor'")
    return sparse_fp8_scaled_linear(xq, xs, w.values, w.meta, w.scale, bias, stream=stream)


# --------------------------------------------------------------------------
# Block-sparse (BSR, 64 x 64 blocks) bf16 weight
# --------------------------------------------------------------------------
BSR_BLOCK = 64


@dataclass
class BsrWeight:
    """A bf16 weight [n, k] in block-sparse form: crow int32 [n/64 + 1], col
    int32 [nnz], values bf16 [nnz, 64, 64] (torch's BSR layout)."""
    crow: torch.Tensor
    col: torch.Tensor
    values: torch.Tensor
    n: int
    k: int

    @property
    def nnz(self) -> int:
        return self.col.shape[0]


def bsr_from_dense(w: torch.Tensor, stream=None) -> BsrWeight:
    """Dense bf16 [n, k] -> BsrWeight keeping every 64 x 64 block that holds a
    non-zero value (two kernels, a read of the block count, one kernel)."""
    _dev(w, "w")
    if w.dtype != torch.bfloat16 or w.dim() != 2:
        raise ValueError("w must be a 2-D bfloat16 tensor")
    n, k = w.shape
    lib, h = load(), _stream(stream)
    crow = torch.empty((n // BSR_BLOCK + 1,), dtype=torch.int32, device=w.device)
    _check(lib.bsr_count_bf16(w.data_ptr(), n, k, crow.data_ptr(), h), "bsr_count_bf16")
    nnz = int(crow[-1].item()) if crow.numel() else 0
    col = torch.empty((nnz,), dtype=torch.int32, device=w.device)
    values = torch.empty((nnz, BSR_BLOCK, BSR_BLOCK), dtype=torch.bfloat16, device=w.device)
    _check(lib.bsr_fill_bf16(w.data_ptr(), n, k, crow.data_ptr(), col.data_ptr() if nnz else None,
                             values.data_ptr() if nnz else None, h), "bsr_fill_bf16")
    return BsrWeight(crow, col, values, n, k)


def bsr_linear(x: torch.Tensor, w: BsrWeight, bias: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """bf16 x [m, k] -> out [m, n] = x @ W^T (+ bias) for the BSR weight W."""
    _dev(x, "x")
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != w.k:
        raise ValueError("x must be bfloat16 [m, k]")
    m = x.shape[0]
    if bias is not None:
        _dev(bias, "bias")
        if bias.dtype != torch.bfloat16 or bias.shape != (w.n,):
            raise ValueError("bias must be bfloat16 [n]")
    od = {torch.bfloat16: SFR_OUT_BF16, torch.float32: SFR_OUT_F32}[out_dtype]
    if out is None:
        out = torch.empty((m, w.n), dtype=out_dtype, device=x.device)
    elif out.shape != (m, w.n) or out.dtype != out_dtype or not out.is_contiguous():
        raise ValueError("out has the wrong shape or dtype")
    _check(load().bsr_linear_bf16(x.data_ptr(), m, w.k, w.crow.data_ptr(), w.col.data_ptr() if w.nnz else None,
                                  w.values.data_ptr() if w.nnz else None, w.n,
                                  None if bias is None else bias.data_ptr(), out.data_ptr(), od, _stream(stream)),
           "bsr_linear_bf16")
    return out


# --------------------------------------------------------------------------
# Gated feed-forward block, MX block formats, 4-bit weights
# --------------------------------------------------------------------------
MX_BLOCK = 32
SFR_ACT = {"silu": 0, "gelu_tanh": 1, "relu": 2}
_BF16 = torch.bfloat16
# None on a torch without these types: the MX formats (scales are E8M0 bytes),
# or their 4-bit form, are then refused as unsupported element types, and
# everything else works.
_E2M1, _E8M0 = getattr(torch, "float4_e2m1fn_x2", None), getattr(torch, "float8_e8m0fnu", None)
_MX = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1} if _E8M0 is not None else {}
_SAVE = {_BF16: 1, **{t: e + 2 for t, e in _MX.items()}}
if _MX and _E2M1 is not None:
    _MX[_E2M1] = 2


@dataclass
class MxTensor:
    """Rows of MX blocks: 32 values along a row share one power-of-two scale.

    codes: float8_e4m3fn or float8_e5m2 [rows, cols], or float4_e2m1fn_x2
    [rows, cols / 2] (two values a byte, the even column in the low half);
    scale: float8_e8m0fnu [rows, cols / 32]."""
    codes: torch.Tensor
    scale: torch.Tensor

    @property
    def shape(self):
        r, c = self.codes.shape
        return (r, 2 * c if self.codes.dtype is _E2M1 else c)


@dataclass
class Int8Tensor:
    """Rows of 8-bit integers with one scale each: codes int8 [rows, cols],
    scale float32 [rows]; a value is scale * code."""
    codes: torch.Tensor
    scale: torch.Tensor

    @property
    def shape(self):
        return tuple(self.codes.shape)


@dataclass
class MoeRoute:
    """A router's choice: ids int32 [m, top] (the experts of every token, best
    first; values outside [0, experts) are no choice), their weights float32
    [m, top], and the logits float32 [m, experts] where moe_route formed them."""
    ids: torch.Tensor
    weights: torch.Tensor
    logits: Optional[torch.Tensor] = None


@dataclass
class GatedCheckpoint:
    """What gated_linear_checkpointed keeps for gated_linear_backward: the
    input x [m, k] and the projections gu = [g | u] [m, 2 f], each a bf16 tensor
    or an 8-bit MxTensor, and the activation's name."""
    x: object
    gu: object
    activation: str


def _current_raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_raw_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _elsewhere(fn, stream, first, *args):
    """fn(first, *args) with first's device current and, with an explicit
    `stream`, with that stream current: what the call allocates then belongs to
    the stream its kernels run on, and the memory of its arguments is not used
    again before that stream is done with them (the stream has to be ordered
    after what produced them, as for any work)."""
    t = first.codes if isinstance(first, (MxTensor, Int8Tensor)) else first
    device = t.get_device()
    if device < 0:
        raise ValueError("the arguments must be GPU tensors")
    if stream is not None and stream.device_index != device:
        raise ValueError(f"stream belongs to GPU {stream.device_index}, the arguments to GPU {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        out = fn(first, *args)
        if stream is not None:
            for a in (first, *args):
                _keep(a, stream)
        return out


def _keep(a, stream):
    """The caching allocator keeps a's memory until `stream` has passed this point."""
    if isinstance(a, torch.Tensor):
        if a.is_cuda:
            a.record_stream(stream)
    elif isinstance(a, (MxTensor, Int8Tensor)):
        _keep(a.codes, stream)
        _keep(a.scale, stream)
    elif isinstance(a, MoeRoute):
        _keep(a.ids, stream)
        _keep(a.weights, stream)
    elif isinstance(a, GatedCheckpoint):
        _keep(a.x, stream)
        _keep(a.gu, stream)


def _refuse(t, name: str, device: int):
    """The reason why t is not a contiguous tensor on GPU `device`."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    if d != device:
        raise ValueError(f"{name} is on GPU {d}, another device than GPU {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _bf16_2d(t: torch.Tensor, name: str, device: int) -> int:
    """t's address, checked."""
    if t.dtype is not _BF16 or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D bfloat16 tensor")
    if t.get_device() != device or device < 0 or not t.is_contiguous():
        _refuse(t, name, device)
    return t.data_ptr()


def _mx_parts(t, name: str, device: int, kinds=_MX):
    """(rows, cols, address of the codes, of the scales) of an MxTensor, checked."""
    if not isinstance(t, MxTensor):
        raise ValueError(f"{name} must be an MxTensor")
    codes, scale = t.codes, t.scale
    dtype = codes.dtype
    if dtype not in kinds:
        raise ValueError(f"{name}: unsupported element type {dtype}")
    if codes.dim() != 2 or scale.dtype is not _E8M0:
        raise ValueError(f"{name}: codes must be 2-D and scale float8_e8m0fnu")
    rows, cols = codes.shape
    if dtype is _E2M1:
        cols *= 2
    if cols % MX_BLOCK != 0 or scale.shape != (rows, cols // MX_BLOCK):
        raise ValueError(f"{name}: scale must have one entry per {MX_BLOCK} columns")
    if codes.get_device() != device or scale.get_device() != device or device < 0 or not codes.is_contiguous() or \
            not scale.is_contiguous():
        _refuse(codes, f"{name}.codes", device)
        _refuse(scale, f"{name}.scale", device)
    return rows, cols, codes.data_ptr(), scale.data_ptr()


def _act_enum(name: str) -> int:
    if name not in SFR_ACT:
        raise ValueError(f"activation must be one of {sorted(SFR_ACT)}")
    return SFR_ACT[name]


def _span(t: torch.Tensor):
    return t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()


def _check_out(out: torch.Tensor, rows: int, cols: int, dtype, *inputs):
    """out has the result's form and overlaps no input."""
    if out.shape != (rows, cols) or out.dtype is not dtype or not out.is_contiguous() or \
            out.device != inputs[0].device:
        raise ValueError("out has the wrong shape, dtype or device")
    start, end = _span(out)
    for t in inputs:
        a, b = _span(t)
        if a < end and start < b:
            raise ValueError("out overlaps an input")


def quantize_mx(x: torch.Tensor, dtype=torch.float8_e4m3fn, *, stream=None) -> MxTensor:
    """bf16 [rows, cols] -> MxTensor of float8_e4m3fn, float8_e5m2 or
    float4_e2m1fn_x2 elements (cols a multiple of 32)."""
    device = x.get_device()
    if stream is not None or device < 0 or device != _current_device():
        return _elsewhere(quantize_mx, stream, x, dtype)
    if dtype not in _MX:
        raise ValueError(f"unsupported element type {dtype}")
    px = _bf16_2d(x, "x", device)
    rows, cols = x.shape
    if cols == 0 or cols % MX_BLOCK != 0:
        raise SfrError(2, "quantize_mx")
    codes = x.new_empty((rows, cols // 2), dtype=dtype) if dtype is _E2M1 else torch.empty_like(x, dtype=dtype)
    scale = x.new_empty((rows, cols // MX_BLOCK), dtype=_E8M0)
    _check(load().quantize_mx(px, rows, cols, _MX[dtype], codes.data_ptr(), scale.data_ptr(), _raw_stream(device)),
           "quantize_mx")
    return MxTensor(codes, scale)


def dequantize_mx(t: MxTensor, out: Optional[torch.Tensor] = None, *, stream=None) -> torch.Tensor:
    """MxTensor -> the bf16 values it stands for (exact for every block that
    quantize_mx writes; the header says what others give)."""
    if not isinstance(t, MxTensor):
        raise ValueError("t must be an MxTensor")
    codes = t.codes
    device = codes.get_device()
    if stream is not None or device < 0 or device != _current_device():
        return _elsewhere(dequantize_mx, stream, t, out)
    rows, cols, pq, ps = _mx_parts(t, "t", device)
    if out is not None:
        _check_out(out, rows, cols, _BF16, codes, t.scale)
    else:
        out = codes.new_empty((rows, cols), dtype=_BF16)
    _check(load().dequantize_mx(pq, ps, rows, cols, _MX[codes.dtype], out.data_ptr(), _raw_stream(device)),
           "dequantize_mx")
    return out


def _gated_operands(x: torch.Tensor, w: torch.Tensor, device: int):
    px, pw = _bf16_2d(x, "x", device), _bf16_2d(w, "w", device)
    m, k = x.shape
    f2, kw = w.shape
    if kw != k or f2 % 2 != 0:
        raise ValueError("w must be [2 f, k] for x [m, k]")
    return px, pw, m, k, f2 // 2


def gated_linear(x: torch.Tensor, w: torch.Tensor, activation: str = "silu", out: Optional[torch.Tensor] = None, *,
                 stream=None) -> torch.Tensor:
    """h [m, f] = act(x @ w[:f].T) * (x @ w[f:].T) for bf16 x [m, k], w [2 f, k].

    The result has no autograd graph, also where x or w require grad; for
    gradients call gated_linear_checkpointed and gated_linear_backward."""
    device = x.get_device()
    if stream is not None or device < 0 or device != _current_device():
        return _elsewhere(gated_linear, stream, x, w, activation, out)
    px, pw, m, k, f = _gated_operands(x, w, device)
    act = _act_enum(activation)
    if out is not None:
        _check_out(out, m, f, _BF16, x, w)
    else:
        out = x.new_empty((m, f))
    _check(load().gated_linear_bf16(px, m, k, pw, f, act, out.data_ptr(), 0, None, None, _raw_stream(device)),
           "gated_linear")
    return out


def gated_linear_checkpointed(x: torch.Tensor, w: torch.Tensor, activation: str = "silu",
                              checkpoint=torch.float8_e4m3fn, *, stream=None):
    """(h, GatedCheckpoint): gated_linear, keeping for the backward pass x and
    the projections in 8 bits (checkpoint float8_e4m3fn or float8_e5m2: MX
    blocks), or x itself and the projections in bf16 (torch.bfloat16).

    h has no autograd graph: hand its gradient to gated_linear_backward."""
    device = x.get_device()
    if stream is not None or device < 0 or device != _current_device():
        return _elsewhere(gated_linear_checkpointed, stream, x, w, activation, checkpoint)
    if checkpoint not in _SAVE:
        raise ValueError(f"unsupported checkpoint type {checkpoint}")
    px, pw, m, k, f = _gated_operands(x, w, device)
    act = _act_enum(activation)
    h = x.new_empty((m, f))
    gu = x.new_empty((m, 2 * f), dtype=checkpoint)
    scale = None if checkpoint is _BF16 else x.new_empty((m, 2 * f // MX_BLOCK), dtype=_E8M0)
    _check(load().gated_linear_bf16(px, m, k, pw, f, act, h.data_ptr(), _SAVE[checkpoint], gu.data_ptr(),
                                    None if scale is None else scale.data_ptr(), _raw_stream(device)),
           "gated_linear_checkpointed")
    if scale is None:
        return h, GatedCheckpoint(x, gu, activation)
    return h, GatedCheckpoint(quantize_mx(x, checkpoint), MxTensor(gu, scale), activation)


def _saved_parts(t, name: str, device: int):
    """(rows, cols, address, address of the scales or None, save enum) of one saved activation."""
    if isinstance(t, MxTensor):
        return (*_mx_parts(t, name, device, _SAVE), _SAVE[t.codes.dtype])
    p = _bf16_2d(t, name, device)
    return (*t.shape, p, None, _SAVE[_BF16])


def gated_linear_backward(dh: torch.Tensor, w: torch.Tensor, saved: GatedCheckpoint, need_dx: bool = True,
                          need_dw: bool = True, *, stream=None):
    """(dx [m, k], dw [2 f, k]) in bf16 from dh [m, f], w and what
    gated_linear_checkpointed kept; None in place of one that is not needed.
    Returned, not added to any .grad."""
    device = dh.get_device()
    if stream is not None or device < 0 or device != _current_device():
        return _elsewhere(gated_linear_backward, stream, dh, w, saved, need_dx, need_dw)
    pd, pw = _bf16_2d(dh, "dh", device), _bf16_2d(w, "w", device)
    xm, xk, px, pxs, x_save = _saved_parts(saved.x, "saved.x", device)
    gm, gf2, pg, pgs, g_save = _saved_parts(saved.gu, "saved.gu", device)
    act = _act_enum(saved.activation)
    m, f = dh.shape
    k = w.shape[1]
    if w.shape[0] != 2 * f or (xm, xk) != (m, k) or (gm, gf2) != (m, 2 * f):
        raise ValueError("operand shapes do not match")
    lib = load()
    dx = dh.new_empty((m, k)) if need_dx else None
    dw = dh.new_empty((2 * f, k)) if need_dw else None
    nbytes = lib.sfr_gated_backward_workspace_bytes(m, k, f, x_save)
    work = dh.new_empty((max(nbytes, 16),), dtype=torch.uint8)
    _check(lib.gated_linear_bf16_backward(pd, m, k, f, act, pg, pgs, g_save, px, pxs, x_save, pw,
                                          dx.data_ptr() if need_dx else None, dw.data_ptr() if need_dw else None,
                                          work.data_ptr(), nbytes, _raw_stream(device)), "gated_linear_backward")
    return dx, dw


_FP4 = tuple(t for t, e in _MX.items() if e == 2)


@functools.lru_cache(maxsize=4096)
def _mxfp4_workspace_bytes(m: int, n: int, k: int) -> int:
    return load().sfr_mxfp4_workspace_bytes(m, n, k)


def _mxfp4_operands(x: torch.Tensor, w: MxTensor, device: int):
    px = _bf16_2d(x, "x", device)
    n, wk, pq, ps = _mx_parts(w, "w", device, _FP4)
    m, k = x.shape
    if wk != k:
        raise ValueError("operand shapes do not match")
    return px, pq, ps, m, n, k


def mxfp4_linear(x: torch.Tensor, w: MxTensor, bias: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                 out: Optional[torch.Tensor] = None, *, stream=None) -> torch.Tensor:
    """bf16 x [m, k] -> out [m, n] = x @ W.T (+ bias) for a 4-bit weight W [n, k]
    with one scale per 32 values, from quantize_mx(w, torch.float4_e2m1fn_x2).
    The result has no autograd graph."""
    device = x.get_device()
    if stream is not None or device < 0 or device != _current_device():
        return _elsewhere(mxfp4_linear, stream, x, w, bias, out_dtype, out)
    px, pq, ps, m, n, k = _mxfp4_operands(x, w, device)
    pb = None
    if bias is not None:
        if bias.dtype is not _BF16 or bias.shape != (n,):
            raise ValueError("bias must be bfloat16 [n]")
        _refuse(bias, "bias", device)
        pb = bias.data_ptr()
    if out_dtype is not _BF16 and out_dtype is not torch.float32:
        raise ValueError("out_dtype must be bfloat16 or float32")
    if out is not None:
        _check_out(out, m, n, out_dtype, x, w.codes, w.scale, *(() if bias is None else (bias,)))
    else:
        out = x.new_empty((m, n), dtype=out_dtype)
    nbytes = _mxfp4_workspace_bytes(m, n, k)
    work = x.new_empty((nbytes,), dtype=torch.uint8) if nbytes else None
    _check(load().mxfp4_linear(px, m, k, pq, ps, n, pb, out.data_ptr(),
                               SFR_OUT_BF16 if out_dtype is _BF16 else SFR_OUT_F32,
                               work.data_ptr() if nbytes else None, nbytes, _raw_stream(device)), "mxfp4_linear")
    return out


def mxfp4_gated_linear(x: torch.Tensor, w: MxTensor, activation: str = "silu", out: Optional[torch.Tensor] = None, *,
                       stream=None) -> torch.Tensor:
    """gated_linear for a 4-bit weight [2 f, k] from quantize_mx(w, torch.float4_e2m1fn_x2).
    The result has no autograd graph."""
    device = x.get_device()
    if stream is not None or device < 0 or device != _current_device():
        return _elsewhere(mxfp4_gated_linear, stream, x, w, activation, out)
    px, pq, ps, m, n, k = _mxfp4_operands(x, w, device)
    act = _act_enum(activation)
    if n % 2 != 0:
        raise ValueError("w must be [2 f, k]")
    if out is not None:
        _check_out(out, m, n // 2, _BF16, x, w.codes, w.scale)
    else:
        out = x.new_empty((m, n // 2))
    _check(load().mxfp4_gated_linear(px, m, k, pq, ps, n // 2, act, out.data_ptr(), _raw_stream(device)),
           "mxfp4_gated_linear")
    return out


_PRODUCTS = {"gated": 0, "gated_saving": 1, "dx": 2, "dw": 3, "mxfp4": 4, "mxfp4_gated": 5}


def block_kernel(product: str, m: int, k: int, f: int):
    """(name, slices of the sum) of the kernel that a product of the block takes:
    "gated" (gated_linear), "gated_saving" (gated_linear_checkpointed), "dx" and
    "dw" (gated_linear_backward), "mxfp4_gated", or "mxfp4" (mxfp4_linear, f its
    n).  None for sizes that the call rejects and for a call without rows."""
    if product not in _PRODUCTS:
        raise ValueError(f"product must be one of {sorted(_PRODUCTS)}")
    slices = ctypes.c_int32()
    name = load().sfr_block_kernel(_PRODUCTS[product], m, k, f, ctypes.byref(slices))
    return None if name is None else (name.decode(), slices.value)


# --------------------------------------------------------------------------
# Linear layer in 8-bit integers
# --------------------------------------------------------------------------
_INT8, _F32, _I32 = torch.int8, torch.float32, torch.int32


def _int8_parts(t, name: str, device: int):
    """(rows, cols, address of the codes, of the scales) of an Int8Tensor, checked."""
    if not isinstance(t, Int8Tensor):
        raise ValueError(f"{name} must be an Int8Tensor")
    codes, scale = t.codes, t.scale
    if codes.dtype is not _INT8 or codes.dim() != 2 or scale.dtype is not _F32:
        raise ValueError(f"{name}: codes must be 2-D int8 and scale float32")
    rows, cols = codes.shape
    if scale.shape != (rows,):
        raise ValueError(f"{name}: scale must have one entry per row")
    if codes.get_device() != device or scale.get_device() != device or device < 0 or not codes.is_contiguous() or \
            not scale.is_contiguous():
        _refuse(codes, f"{name}.codes", device)
        _refuse(scale, f"{name}.scale", device)
    return rows, cols, codes.data_ptr(), scale.data_ptr()


def quantize_rowwise_int8(x: torch.Tensor, *, stream=None) -> Int8Tensor:
    """bf16 [rows, cols] -> Int8Tensor, scale = amax / 127 for every row: an
    activation by token, or a weight [n, k] by output channel (cols a multiple of 8)."""
    device = x.get_device()
    if stream is not None or device < 0 or device != _current_device():
        return _elsewhere(quantize_rowwise_int8, stream, x)
    px = _bf16_2d(x, "x", device)
    rows, cols = x.shape
    codes = torch.empty_like(x, dtype=_INT8)
    scale = x.new_empty((rows,), dtype=_F32)
    _check(load().quantize_rowwise_int8(px, rows, cols, codes.data_ptr(), scale.data_ptr(), _raw_stream(device)),
           "quantize_rowwise_int8")
    return Int8Tensor(codes, scale)


@functools.lru_cache(maxsize=4096)
def _int8_workspace_bytes(m: int, n: int, k: int, dynamic: bool) -> int:
    return load().sfr_int8_workspace_bytes(m, n, k, dynamic)


def int8_linear(x, w: Int8Tensor, bias: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                out: Optional[torch.Tensor] = None, *, stream=None) -> torch.Tensor:
    """x [m, k] -> out [m, n] = x @ W.T (+ bias) in 8-bit integers for a weight W
    [n, k] from quantize_rowwise_int8.  x: bf16, quantized by token in the call,
    or an Int8Tensor (one quantization for several products); both give the same
    bits.  The result has no autograd graph."""
    dynamic = not isinstance(x, Int8Tensor)
    first = x if dynamic else x.codes
    device = first.get_device()
    if stream is not None or device < 0 or device != _current_device():
        return _elsewhere(int8_linear, stream, x, w, bias, out_dtype, out)
    if dynamic:
        px = _bf16_2d(x, "x", device)
        m, k = x.shape
    else:
        m, k, px, pxs = _int8_parts(x, "x", device)
    n, wk, pw, pws = _int8_parts(w, "w", device)
    if wk != k:
        raise ValueError("operand shapes do not match")
    pb = None
    if bias is not None:
        if bias.dtype is not _BF16 or bias.shape != (n,):
            raise ValueError("bias must be bfloat16 [n]")
        _refuse(bias, "bias", device)
        pb = bias.data_ptr()
    if out_dtype is not _BF16 and out_dtype is not _F32:
        raise ValueError("out_dtype must be bfloat16 or float32")
    if out is not None:
        _check_out(out, m, n, out_dtype, first, w.codes, w.scale, *(() if dynamic else (x.scale,)),
                   *(() if bias is None else (bias,)))
    else:
        out = w.scale.new_empty((m, n), dtype=out_dtype)
    od = SFR_OUT_BF16 if out_dtype is _BF16 else SFR_OUT_F32
    nbytes = _int8_workspace_bytes(m, n, k, dynamic)
    work = w.codes.new_empty((nbytes,)) if nbytes else None
    pwork = work.data_ptr() if nbytes else None
    if dynamic:
        _check(load().int8_linear_dynamic(px, m, k, pw, pws, n, pb, out.data_ptr(), od, pwork, nbytes,
                                          _raw_stream(device)), "int8_linear")
    else:
        _check(load().int8_scaled_linear(px, pxs, m, k, pw, pws, n, pb, out.data_ptr(), od, pwork, nbytes,
                                         _raw_stream(device)), "int8_linear")
    return out


def int8_kernel(m: int, n: int, k: int, dynamic: bool = True):
    """(name, slices of the sum) of the kernel that int8_linear's product takes, as
    block_kernel gives it; None for sizes that the call rejects or that leave nothing to do."""
    slices = ctypes.c_int32()
    name = load().sfr_int8_kernel(m, n, k, dynamic, ctypes.byref(slices))
    return None if name is None else (name.decode(), slices.value)


# --------------------------------------------------------------------------
# Mixture of gated feed-forward blocks for a few tokens
# --------------------------------------------------------------------------
SFR_ROUTE = {"softmax": 0, "sigmoid": 1}


def moe_route(x: torch.Tensor, w: torch.Tensor, top: int, bias: Optional[torch.Tensor] = None,
              score: str = "softmax", renormalize: bool = True, *, stream=None) -> MoeRoute:
    """The `top` best experts of every token: logits = x @ w.T (+ bias) for bf16 x
    [m, k], w [experts, k] and float32 bias [experts]; weights from their softmax
    over all experts or their sigmoid, divided by the chosen ones' sum with
    `renormalize`.  Of equal logits the lowest expert comes first; an expert whose
    bias is -inf is never chosen (a slot left over: id -1, weight 0).  The logits'
    sum is formed in binary64, so the choice does not depend on the rest of the
    batch.  The results have no autograd graph."""
    device = x.get_device()
    if stream is not None or device < 0 or device != _current_device():
        return _elsewhere(moe_route, stream, x, w, top, bias, score, renormalize)
    px, pw = _bf16_2d(x, "x", device), _bf16_2d(w, "w", device)
    m, k = x.shape
    experts, wk = w.shape
    if wk != k:
        raise ValueError("operand shapes do not match")
    if score not in SFR_ROUTE:
        raise ValueError(f"score must be one of {sorted(SFR_ROUTE)}")
    pb = None
    if bias is not None:
        if bias.dtype is not _F32 or bias.shape != (experts,):
            raise ValueError("bias must be float32 [experts]")
        _refuse(bias, "bias", device)
        pb = bias.data_ptr()
    if not 0 < top <= experts:
        raise ValueError("top must be between 1 and the number of experts")
    logits = x.new_empty((m, experts), dtype=_F32)
    ids = x.new_empty((m, top), dtype=_I32)
    weights = x.new_empty((m, top), dtype=_F32)
    _check(load().moe_route(px, m, k, pw, experts, pb, top, SFR_ROUTE[score], renormalize, logits.data_ptr(),
                            ids.data_ptr(), weights.data_ptr(), _raw_stream(device)), "moe_route")
    return MoeRoute(ids, weights, logits)


def _expert_parts(t, name: str, device: int):
    """(form, rows, cols, address of the weights, of the scales or None) of the
    experts' stacked weight rows, checked."""
    if isinstance(t, Int8Tensor):
        return (1, *_int8_parts(t, name, device))
    if isinstance(t, MxTensor):
        return (2, *_mx_parts(t, name, device, _FP4))
    if not isinstance(t, torch.Tensor) or t.dtype is not _BF16 or t.dim() != 3:
        raise ValueError(f"{name} must be a 3-D bfloat16 tensor, an Int8Tensor or a 4-bit MxTensor")
    if t.get_device() != device or device < 0 or not t.is_contiguous():
        _refuse(t, name, device)
    a, b, c = t.shape
    return 0, a * b, c, t.data_ptr(), None


@functools.lru_cache(maxsize=4096)
def _moe_workspace_bytes(m: int, k: int, f: int, top: int) -> int:
    return load().sfr_moe_workspace_bytes(m, k, f, top)


def moe_layer(x: torch.Tensor, route: MoeRoute, w_gate_up, w_down, activation: str = "silu",
              out: Optional[torch.Tensor] = None, *, stream=None) -> torch.Tensor:
    """The whole mixture of gated feed-forward blocks for a few tokens:
    out[t] = sum_s weights[t, s] * (act(x[t] @ Wg[e].T) * (x[t] @ Wu[e].T)) @ Wd[e].T,
    e = ids[t, s], for bf16 x [m, k].

    w_gate_up: bf16 [experts, 2 f, k], every expert's gate rows and then its up
    rows; or those rows stacked [experts * 2 f, k] in 8 bits
    (quantize_rowwise_int8) or 4 bits (quantize_mx(w, torch.float4_e2m1fn_x2)).
    w_down: bf16 [experts, k, f], or stacked [experts * k, f] in the same form.
    Tokens are taken 64 at a time, each time reading the chosen experts' weights
    once.  ids outside [0, experts) are no choice; a token without one gets zeros.
    The result has no autograd graph."""
    device = x.get_device()
    if stream is not None or device < 0 or device != _current_device():
        return _elsewhere(moe_layer, stream, x, route, w_gate_up, w_down, activation, out)
    px = _bf16_2d(x, "x", device)
    m, k = x.shape
    ids, weights = route.ids, route.weights
    if ids.dtype is not _I32 or weights.dtype is not _F32 or ids.dim() != 2 or ids.shape[0] != m or \
            weights.shape != ids.shape:
        raise ValueError("route must hold ids int32 [m, top] and weights float32 [m, top]")
    if ids.get_device() != device or weights.get_device() != device or not ids.is_contiguous() or \
            not weights.is_contiguous():
        _refuse(ids, "route.ids", device)
        _refuse(weights, "route.weights", device)
    form, rows, wk, pg, pgs = _expert_parts(w_gate_up, "w_gate_up", device)
    dform, drows, f, pd, pds = _expert_parts(w_down, "w_down", device)
    experts = drows // k if k else 0
    if dform != form:
        raise ValueError("w_gate_up and w_down must be of the same form")
    if wk != k or experts * k != drows or experts * 2 * f != rows or \
            form == 0 and not (w_gate_up.shape[0] == w_down.shape[0] == experts):
        raise ValueError("operand shapes do not match: w_gate_up [experts, 2 f, k], w_down [experts, k, f]")
    act = _act_enum(activation)
    if out is not None:
        parts = [t for w in (w_gate_up, w_down) for t in ((w,) if form == 0 else (w.codes, w.scale))]
        _check_out(out, m, k, _BF16, x, ids, weights, *parts)
    else:
        out = torch.empty_like(x)
    top = ids.shape[1]
    nbytes = _moe_workspace_bytes(m, k, f, top)
    work = x.new_empty((nbytes // 2 + 8,))  # bf16
    _check(load().moe_layer(px, m, k, ids.data_ptr(), weights.data_ptr(), top, experts, f, form, pg, pgs, pd, pds, act,
                         out.data_ptr(), work.data_ptr(), nbytes, _raw_stream(device)), "moe_layer")
    return out
