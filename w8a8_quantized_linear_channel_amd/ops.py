"""Thin torch binding of the libq8 C ABI, one Python function per C call and
with the same name.  It checks tensor devices/dtypes/shapes, allocates
outputs and the workspace with torch, passes raw device pointers and the
current HIP stream, and turns a non-OK status into an exception.  All
arithmetic happens in the HIP kernels."""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional

import torch

from . import _lib

_DT = {torch.float32: _lib.Q8_F32, torch.float16: _lib.Q8_F16, torch.bfloat16: _lib.Q8_BF16}
_FMT = {"int8_asym": _lib.Q8_INT8_ASYM, "int8_sym": _lib.Q8_INT8_SYM, "fp8_e4m3": _lib.Q8_FP8_E4M3}
_OP = {"linear": _lib.Q8_OP_LINEAR, "decomp": _lib.Q8_OP_DECOMP, "fp8": _lib.Q8_OP_FP8,
       "static": _lib.Q8_OP_STATIC, "grouped": _lib.Q8_OP_GROUPED, "fp8_block": _lib.Q8_OP_FP8_BLOCK}


class _DtypeCodes(dict):
    """torch dtype -> q8_dtype code; an unsupported dtype is a TypeError that
    names the supported ones."""

    def __missing__(self, key):
        raise TypeError(f"unsupported dtype {key}: expected torch.float32, torch.float16 or torch.bfloat16")


_DT = _DtypeCodes(_DT)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(dev: torch.device) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


def _need(t: torch.Tensor, name: str, dtype=None, shape=None, dev=None) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")


def q8_workspace_bytes(op: str, M: int, N: int, K: int) -> int:
    return int(_lib.lib().q8_workspace_bytes(_OP[op], M, N, K))


def _workspace(op: str, M: int, N: int, K: int, dev, given: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The caller's workspace, checked (the call checks its size), or one of the size that the call needs."""
    if given is not None:
        _need(given, "workspace", None, None, dev)
        return given
    n = q8_workspace_bytes(op, M, N, K)
    return torch.empty(max(n, 1), dtype=torch.uint8, device=dev)


def q8_quantize_weight(w: torch.Tensor, fmt: str = "int8_asym"):
    """Per-output-channel weight quantization.  Returns (wq, scale, zero_point);
    zero_point is None for "fp8_e4m3" (codes are returned as uint8)."""
    _need(w, "w")
    if w.dim() != 2 or w.dtype not in _DT:
        raise ValueError("w must be 2-D float32/float16/bfloat16")
    N, K = w.shape
    dev = w.device
    if fmt == "int8_asym":
        wq = torch.empty(N, K, dtype=torch.int8, device=dev)
        zp = torch.empty(N, dtype=torch.float32, device=dev)
    elif fmt == "fp8_e4m3":
        wq = torch.empty(N, K, dtype=torch.uint8, device=dev)
        zp = None
    else:
        raise ValueError(f"unsupported weight format {fmt}")
    scale = torch.empty(N, dtype=torch.float32, device=dev)
    st = _lib.lib().q8_quantize_weight(_FMT[fmt], _ptr(w), _DT[w.dtype], N, K, _ptr(wq), _ptr(scale),
                                       _ptr(zp), _stream(dev))
    _lib.check("q8_quantize_weight", st)
    return wq, scale, zp


def q8_quantize_act(x: torch.Tensor, fmt: str = "int8_sym", scale_ub: float = math.inf,
                    rowsum: bool = True, out=None):
    """Dynamic per-token quantization.  Returns (xq, scale, rowsum or None);
    `out` may supply those three tensors preallocated."""
    _need(x, "x")
    if x.dim() != 2 or x.dtype not in _DT:
        raise ValueError("x must be 2-D float32/float16/bfloat16")
    M, K = x.shape
    dev = x.device
    if fmt not in ("int8_sym", "fp8_e4m3"):
        raise ValueError(f"unsupported activation format {fmt}")
    code_dt = torch.int8 if fmt == "int8_sym" else torch.uint8
    if out is not None:
        xq, scale, rs = out
        _need(xq, "xq", code_dt, (M, K), dev)
        _need(scale, "scale", torch.float32, (M,), dev)
        if rs is not None:
            _need(rs, "rowsum", torch.int32, (M,), dev)
    else:
        xq = torch.empty(M, K, dtype=code_dt, device=dev)
        scale = torch.empty(M, dtype=torch.float32, device=dev)
        rs = torch.empty(M, dtype=torch.int32, device=dev) if (rowsum and fmt == "int8_sym") else None
    st = _lib.lib().q8_quantize_act(_FMT[fmt], _ptr(x), _DT[x.dtype], M, K, float(scale_ub), _ptr(xq),
                                    _ptr(scale), _ptr(rs), _stream(dev))
    _lib.check("q8_quantize_act", st)
    return xq, scale, rs


def q8_linear(x: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor, w_zp: torch.Tensor,
              bias: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
              acc_out: bool = False, workspace: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None):
    """W8A8 linear.  Returns y (and the INT32 accumulator if acc_out)."""
    _need(x, "x")
    dev = x.device
    M, K = x.shape
    N = wq.shape[0]
    _need(wq, "wq", torch.int8, (N, K), dev)
    _need(w_scale, "w_scale", torch.float32, (N,), dev)
    _need(w_zp, "w_zp", torch.float32, (N,), dev)
    if bias is not None:
        _need(bias, "bias", torch.float32, (N,), dev)
    out_dtype = out_dtype or x.dtype
    y = out if out is not None else torch.empty(M, N, dtype=out_dtype, device=dev)
    _need(y, "y", out_dtype, (M, N), dev)
    acc = torch.empty(M, N, dtype=torch.int32, device=dev) if acc_out else None
    ws = _workspace("linear", M, N, K, dev, workspace)
    st = _lib.lib().q8_linear(_ptr(x), _DT[x.dtype], M, K, _ptr(wq), _ptr(w_scale), _ptr(w_zp), N,
                              _ptr(bias), _ptr(y), _DT[out_dtype], _ptr(ws), ws.nbytes, _ptr(acc),
                              _stream(dev))
    _lib.check("q8_linear", st)
    return (y, acc) if acc_out else y


def q8_linear_noalloc(x: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor, w_zp: torch.Tensor,
                      bias: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                      acc_out: bool = False, out: Optional[torch.Tensor] = None):
    """q8_linear without a workspace (the library's own scratch array); with
    `out` (and acc_out False) the binding allocates nothing either.  Returns y
    (and the INT32 accumulator if acc_out)."""
    _need(x, "x")
    dev = x.device
    M, K = x.shape
    N = wq.shape[0]
    _need(wq, "wq", torch.int8, (N, K), dev)
    _need(w_scale, "w_scale", torch.float32, (N,), dev)
    _need(w_zp, "w_zp", torch.float32, (N,), dev)
    if bias is not None:
        _need(bias, "bias", torch.float32, (N,), dev)
    out_dtype = out_dtype or x.dtype
    y = out if out is not None else torch.empty(M, N, dtype=out_dtype, device=dev)
    _need(y, "y", out_dtype, (M, N), dev)
    acc = torch.empty(M, N, dtype=torch.int32, device=dev) if acc_out else None
    st = _lib.lib().q8_linear_noalloc(_ptr(x), _DT[x.dtype], M, K, _ptr(wq), _ptr(w_scale), _ptr(w_zp), N,
                                      _ptr(bias), _ptr(y), _DT[out_dtype], _ptr(acc), _stream(dev))
    _lib.check("q8_linear_noalloc", st)
    return (y, acc) if acc_out else y


def q8_linear_int8_decomp(x: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor,
                          w_zp: torch.Tensor, threshold: float = 6.0,
                          bias: Optional[torch.Tensor] = None, return_outliers: bool = False,
                          acc_out: bool = False, workspace: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None):
    """LLM.int8() decomposition.  Returns y, plus (outlier_idx, n_outliers)
    device tensors if return_outliers, plus the int8-path accumulator if acc_out."""
    _need(x, "x", torch.float16)
    dev = x.device
    M, K = x.shape
    N = wq.shape[0]
    _need(wq, "wq", torch.int8, (N, K), dev)
    _need(w_scale, "w_scale", torch.float32, (N,), dev)
    _need(w_zp, "w_zp", torch.float32, (N,), dev)
    if bias is not None:
        _need(bias, "bias", torch.float32, (N,), dev)
    y = out if out is not None else torch.empty(M, N, dtype=torch.float16, device=dev)
    _need(y, "y", torch.float16, (M, N), dev)
    idx = torch.empty(K, dtype=torch.int32, device=dev) if return_outliers else None
    cnt = torch.empty(1, dtype=torch.int32, device=dev) if return_outliers else None
    acc = torch.empty(M, N, dtype=torch.int32, device=dev) if acc_out else None
    ws = _workspace("decomp", M, N, K, dev, workspace)
    st = _lib.lib().q8_linear_int8_decomp(_ptr(x), M, K, _ptr(wq), _ptr(w_scale), _ptr(w_zp), N,
                                          float(threshold), _ptr(bias), _ptr(y), _ptr(ws), ws.nbytes,
                                          _ptr(idx), _ptr(cnt), _ptr(acc), _stream(dev))
    _lib.check("q8_linear_int8_decomp", st)
    res = [y]
    if return_outliers:
        res += [idx, cnt]
    if acc_out:
        res.append(acc)
    return res[0] if len(res) == 1 else tuple(res)


def q8_linear_fp8(x: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor,
                  scale_ub: float = 1200.0, bias: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """FP8 e4m3 W8A8 rowwise linear (bf16 in, bf16 out)."""
    _need(x, "x", torch.bfloat16)
    dev = x.device
    M, K = x.shape
    N = wq.shape[0]
    _need(wq, "wq", torch.uint8, (N, K), dev)
    _need(w_scale, "w_scale", torch.float32, (N,), dev)
    if bias is not None:
        _need(bias, "bias", torch.float32, (N,), dev)
    y = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    _need(y, "y", torch.bfloat16, (M, N), dev)
    ws = _workspace("fp8", M, N, K, dev, workspace)
    st = _lib.lib().q8_linear_fp8(_ptr(x), M, K, _ptr(wq), _ptr(w_scale), N, float(scale_ub), _ptr(bias),
                                  _ptr(y), _ptr(ws), ws.nbytes, _stream(dev))
    _lib.check("q8_linear_fp8", st)
    return y


def q8_gemm_int8(xq: torch.Tensor, x_scale: torch.Tensor, x_rowsum: torch.Tensor, wq: torch.Tensor,
                 w_scale: torch.Tensor, w_zp: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 out_dtype: torch.dtype = torch.bfloat16, acc_out: bool = False,
                 out: Optional[torch.Tensor] = None):
    """INT8 GEMM + dequantization epilogue on pre-quantized activations."""
    _need(xq, "xq", torch.int8)
    dev = xq.device
    M, K = xq.shape
    N = wq.shape[0]
    _need(x_scale, "x_scale", torch.float32, (M,), dev)
    _need(x_rowsum, "x_rowsum", torch.int32, (M,), dev)
    _need(wq, "wq", torch.int8, (N, K), dev)
    _need(w_scale, "w_scale", torch.float32, (N,), dev)
    _need(w_zp, "w_zp", torch.float32, (N,), dev)
    if bias is not None:
        _need(bias, "bias", torch.float32, (N,), dev)
    y = out if out is not None else torch.empty(M, N, dtype=out_dtype, device=dev)
    _need(y, "y", out_dtype, (M, N), dev)
    acc = torch.empty(M, N, dtype=torch.int32, device=dev) if acc_out else None
    st = _lib.lib().q8_gemm_int8(_ptr(xq), _ptr(x_scale), _ptr(x_rowsum), M, K, _ptr(wq), _ptr(w_scale),
                                 _ptr(w_zp), N, _ptr(bias), _ptr(y), _DT[out_dtype], _ptr(acc),
                                 _stream(dev))
    _lib.check("q8_gemm_int8", st)
    return (y, acc) if acc_out else y


def q8_gemm_fp8(xq: torch.Tensor, x_scale: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor,
                bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """Rowwise FP8 GEMM on e4m3 codes (bf16 out)."""
    _need(xq, "xq", torch.uint8)
    dev = xq.device
    M, K = xq.shape
    N = wq.shape[0]
    _need(x_scale, "x_scale", torch.float32, (M,), dev)
    _need(wq, "wq", torch.uint8, (N, K), dev)
    _need(w_scale, "w_scale", torch.float32, (N,), dev)
    if bias is not None:
        _need(bias, "bias", torch.float32, (N,), dev)
    y = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    _need(y, "y", torch.bfloat16, (M, N), dev)
    st = _lib.lib().q8_gemm_fp8(_ptr(xq), _ptr(x_scale), M, K, _ptr(wq), _ptr(w_scale), N, _ptr(bias),
                                _ptr(y), _stream(dev))
    _lib.check("q8_gemm_fp8", st)
    return y


def q8_linear_w8a16(x: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor, w_zp: torch.Tensor,
                    bias: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                    out: Optional[torch.Tensor] = None):
    """Weight-only W8A16 linear for up to 16 tokens: y = x . (S_w (Wq - Z_w))^T (+ bias),
    x bf16 or fp16, weights from q8_quantize_weight("int8_asym")."""
    dev = x.device
    M, K = x.shape
    N = wq.shape[0]
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("q8_linear_w8a16: x must be bfloat16 or float16")
    _need(x, "x", x.dtype, (M, K), dev)
    _need(wq, "wq", torch.int8, (N, K), dev)
    _need(w_scale, "w_scale", torch.float32, (N,), dev)
    _need(w_zp, "w_zp", torch.float32, (N,), dev)
    if bias is not None:
        _need(bias, "bias", torch.float32, (N,), dev)
    y = out if out is not None else torch.empty(M, N, dtype=out_dtype, device=dev)
    _need(y, "y", out_dtype, (M, N), dev)
    st = _lib.lib().q8_linear_w8a16(_ptr(x), _DT[x.dtype], M, K, _ptr(wq), _ptr(w_scale), _ptr(w_zp), N,
                                    _ptr(bias), _ptr(y), _DT[out_dtype], _stream(dev))
    _lib.check("q8_linear_w8a16", st)
    return y


def q8_quantize_act_static(x: torch.Tensor, x_scale: float, out=None):
    """Static INT8 codes with one calibrated scale: (xq int8 [M,K], rowsum int32 [M])."""
    dev = x.device
    M, K = x.shape
    _need(x, "x", x.dtype, (M, K), dev)
    xq, rs = out if out is not None else (torch.empty(M, K, dtype=torch.int8, device=dev),
                                          torch.empty(M, dtype=torch.int32, device=dev))
    _need(xq, "xq", torch.int8, (M, K), dev)
    _need(rs, "x_rowsum", torch.int32, (M,), dev)
    st = _lib.lib().q8_quantize_act_static(_ptr(x), _DT[x.dtype], M, K, float(x_scale), _ptr(xq), _ptr(rs),
                                           _stream(dev))
    _lib.check("q8_quantize_act_static", st)
    return xq, rs


def q8_linear_static(x: torch.Tensor, x_scale: float, wq: torch.Tensor, w_scale: torch.Tensor,
                     w_zp: torch.Tensor, y_scale: float, bias: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """W8A8 linear with a static activation scale and INT8 output codes (scale y_scale)."""
    dev = x.device
    M, K = x.shape
    N = wq.shape[0]
    _need(x, "x", x.dtype, (M, K), dev)
    _need(wq, "wq", torch.int8, (N, K), dev)
    _need(w_scale, "w_scale", torch.float32, (N,), dev)
    _need(w_zp, "w_zp", torch.float32, (N,), dev)
    if bias is not None:
        _need(bias, "bias", torch.float32, (N,), dev)
    yq = out if out is not None else torch.empty(M, N, dtype=torch.int8, device=dev)
    _need(yq, "yq", torch.int8, (M, N), dev)
    ws = _workspace("static", M, N, K, dev, workspace)
    st = _lib.lib().q8_linear_static(_ptr(x), _DT[x.dtype], M, K, float(x_scale), _ptr(wq), _ptr(w_scale),
                                     _ptr(w_zp), N, _ptr(bias), float(y_scale), _ptr(yq), _ptr(ws),
                                     ws.nbytes, _stream(dev))
    _lib.check("q8_linear_static", st)
    return yq


def q8_linear_fp8_grouped(x: torch.Tensor, expert_offsets: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor,
                          scale_ub: float = 1200.0, out: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None):
    """FP8 expert projection on routed tokens: x bf16 [T,K] grouped by expert,
    expert_offsets int32 [E+1] on the device, wq e4m3 [E,N,K], w_scale [E,N]."""
    _need(x, "x", torch.bfloat16)
    dev = x.device
    T, K = x.shape
    E, N = wq.shape[0], wq.shape[1]
    _need(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev)
    _need(wq, "wq", torch.uint8, (E, N, K), dev)
    _need(w_scale, "w_scale", torch.float32, (E, N), dev)
    y = out if out is not None else torch.empty(T, N, dtype=torch.bfloat16, device=dev)
    _need(y, "y", torch.bfloat16, (T, N), dev)
    ws = _workspace("fp8", T, N, K, dev, workspace)
    st = _lib.lib().q8_linear_fp8_grouped(_ptr(x), T, K, _ptr(expert_offsets), E, _ptr(wq), _ptr(w_scale), N,
                                          float(scale_ub), _ptr(y), _ptr(ws), ws.nbytes, _stream(dev))
    _lib.check("q8_linear_fp8_grouped", st)
    return y


def q8_quantize_weight_grouped(w: torch.Tensor, group: int = 128):
    """Per-group asymmetric INT8 weights: returns (wq int8 [N, K], w_scale float32
    [K/group, N], w_zp float32 [K/group, N]), the parameters group-major."""
    dev = w.device
    N, K = w.shape
    if w.dtype not in _DT:
        raise TypeError(f"q8_quantize_weight_grouped: unsupported dtype {w.dtype}")
    _need(w, "w", w.dtype, (N, K), dev)
    G = K // group if group > 0 else 0
    wq = torch.empty(N, K, dtype=torch.int8, device=dev)
    ws = torch.empty(max(G, 1), N, dtype=torch.float32, device=dev)
    wz = torch.empty(max(G, 1), N, dtype=torch.float32, device=dev)
    st = _lib.lib().q8_quantize_weight_grouped(_ptr(w), _DT[w.dtype], N, K, group, _ptr(wq), _ptr(ws), _ptr(wz),
                                               _stream(dev))
    _lib.check("q8_quantize_weight_grouped", st)
    return wq, ws, wz


def q8_linear_grouped(x: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor, w_zp: torch.Tensor,
                      group: int = 128, bias: Optional[torch.Tensor] = None,
                      out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None):
    """W8A8 linear with per-group weights (from q8_quantize_weight_grouped with the
    same group) and dynamic per-token INT8 activations."""
    dev = x.device
    M, K = x.shape
    N = wq.shape[0]
    G = K // group if group > 0 else 0
    _need(x, "x", x.dtype, (M, K), dev)
    _need(wq, "wq", torch.int8, (N, K), dev)
    _need(w_scale, "w_scale", torch.float32, (G, N), dev)
    _need(w_zp, "w_zp", torch.float32, (G, N), dev)
    if bias is not None:
        _need(bias, "bias", torch.float32, (N,), dev)
    y = out if out is not None else torch.empty(M, N, dtype=out_dtype, device=dev)
    _need(y, "y", out_dtype, (M, N), dev)
    ws = _workspace("grouped", M, N, K, dev, workspace)
    st = _lib.lib().q8_linear_grouped(_ptr(x), _DT[x.dtype], M, K, _ptr(wq), _ptr(w_scale), _ptr(w_zp), group, N,
                                      _ptr(bias), _ptr(y), _DT[out_dtype], _ptr(ws), ws.nbytes, _stream(dev))
    _lib.check("q8_linear_grouped", st)
    return y


class KvCache(NamedTuple):
    """The paged 8-bit key/value cache of one layer: e4m3 codes of the keys
    [pages, kv_heads, page, dim] and of the values [pages, kv_heads, dim, page],
    and an exponent byte b per page and head [pages, kv_heads] (a code c stands
    for e4m3(c) * 2^(b - 127)).  One-byte dtypes: uint8, or float8_e4m3fn for
    codes and float8_e8m0fnu for exponents."""
    k: torch.Tensor
    k_exp: torch.Tensor
    v: torch.Tensor
    v_exp: torch.Tensor


class KvBatch(NamedTuple):
    """The sequences of one call over a KvCache: new tokens q_start[s] ..
    q_start[s+1]-1 belong to sequence s, whose length with them is kv_len[s] and
    whose pages are block_table[s] (int32 device tensors [S+1], [S] and
    [S, max_pages]); max_q and max_kv bound the new tokens and the length of one
    sequence (a bound that is too small costs time, not results)."""
    q_start: torch.Tensor
    kv_len: torch.Tensor
    block_table: torch.Tensor
    max_q: int
    max_kv: int


def q8_kv_cache(num_pages: int, kv_heads: int, head_dim: int, page: int = 64, device="cuda") -> KvCache:
    """An empty cache (all bytes zero)."""
    z = lambda *shape: torch.zeros(*shape, dtype=torch.uint8, device=device)  # noqa: E731
    return KvCache(z(num_pages, kv_heads, page, head_dim), z(num_pages, kv_heads),
                   z(num_pages, kv_heads, head_dim, page), z(num_pages, kv_heads))


_CODES = (torch.uint8, torch.float8_e4m3fn)      # of e4m3 codes
_EXPS = (torch.uint8, torch.float8_e8m0fnu)
_I32 = torch.int32


def _raw_stream(index: int) -> int:
    """The current stream of device `index` as a raw handle (without building a Stream object)."""
    return torch._C._cuda_getCurrentRawStream(index)


_FAST = None


def _fast():
    """The compiled half of this binding (binding.cpp), which does the checks and the call of the
    latency-bound functions; a result of NotImplemented means an argument it does not take, and the
    checks below say what is wrong with it."""
    global _FAST
    if _FAST is None:
        _lib.lib()                      # says how to build what is missing
        from . import _binding
        _FAST = _binding
    return _FAST


def _result(func: str, r):
    """A compiled call's result, or its C status as an exception."""
    if type(r) is int:
        _lib.check(func, r)
    return r


def _is(t, dtype, shape, index: int) -> bool:
    """A dense tensor of this dtype and shape on device `index` (the check of the calls whose
    latency counts; _need says what is wrong where this is False)."""
    return t.get_device() == index and t.dtype is dtype and t.shape == shape and t.is_contiguous()


def _check_kv(cache: KvCache, batch: KvBatch, dev, index: int):
    """Checks a cache and a batch over it; returns (pages, kv_heads, page, dim, seqs, max_pages)."""
    k, ke, v, ve = cache
    start, lens, table, _, _ = batch
    if k.dim() == 4 and table.dim() == 2:
        P, Hkv, page, D = shape = k.shape
        S, max_pages = tshape = table.shape
        cd, ed = k.dtype, ke.dtype
        if (cd in _CODES and ed in _EXPS and _is(k, cd, shape, index) and _is(v, cd, (P, Hkv, D, page), index)
                and _is(ke, ed, (P, Hkv), index) and _is(ve, ed, (P, Hkv), index) and _is(table, _I32, tshape, index)
                and _is(start, _I32, (S + 1,), index) and _is(lens, _I32, (S,), index)):
            return P, Hkv, page, D, S, max_pages
    # something is wrong: say what
    if k.dim() != 4 or k.dtype not in _CODES:
        raise ValueError("cache.k must be 4-D uint8 or float8_e4m3fn")
    if ke.dtype not in _EXPS:
        raise TypeError(f"cache.k_exp must be uint8 or float8_e8m0fnu, got {ke.dtype}")
    if table.dim() != 2:
        raise ValueError("batch.block_table must be 2-D")
    P, Hkv, page, D = k.shape
    S = table.shape[0]
    _need(k, "cache.k", k.dtype, None, dev)
    _need(v, "cache.v", k.dtype, (P, Hkv, D, page), dev)
    _need(ke, "cache.k_exp", ke.dtype, (P, Hkv), dev)
    _need(ve, "cache.v_exp", ke.dtype, (P, Hkv), dev)
    _need(table, "batch.block_table", _I32, None, dev)
    _need(start, "batch.q_start", _I32, (S + 1,), dev)
    _need(lens, "batch.kv_len", _I32, (S,), dev)
    raise ValueError("unsupported cache or batch")


def _rows(t: torch.Tensor, name: str, dtype, tail, index: int) -> int:
    """Checks a [tokens, heads, dim] tensor, heads and features dense, tokens any stride apart;
    returns that stride."""
    if t.get_device() != index:
        raise (TypeError(f"{name} must be a CUDA (HIP) tensor") if not t.is_cuda else
               ValueError(f"{name} is on {t.device}, expected cuda:{index}"))
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or t.shape[1:] != tail:
        raise ValueError(f"{name} must have shape [tokens, {tail[0]}, {tail[1]}], got {tuple(t.shape)}")
    step, heads, one = t.stride()
    if (one != 1 or (heads != tail[1] and tail[0] > 1)) and t.numel():
        raise ValueError(f"{name} must have dense heads and features")
    return step


def _cuda_index(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    return t.get_device()


def q8_kv_append(k: torch.Tensor, v: torch.Tensor, cache: KvCache, batch: KvBatch,
                 q: Optional[torch.Tensor] = None, cos: Optional[torch.Tensor] = None,
                 sin: Optional[torch.Tensor] = None, interleaved: bool = False,
                 out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Put the new keys and values [T, kv_heads, dim] into the cache (in place),
    keys rotated by cos, sin [positions, rot_dim / 2] if given; returns the
    rotated queries of q [T, heads, dim], or None without q.  k, v and q may be
    slices of one projection's output (any token stride)."""
    r = _fast().kv_append(k, v, cache, batch, q, cos, sin, interleaved, out)
    if r is not NotImplemented:
        return _result("q8_kv_append", r)
    index, dev = _cuda_index(k, "k"), k.device
    P, Hkv, page, D, S, max_pages = _check_kv(cache, batch, dev, index)
    dt = k.dtype
    k_step = _rows(k, "k", dt, (Hkv, D), index)
    v_step = _rows(v, "v", dt, (Hkv, D), index)
    T = k.shape[0]
    if v.shape[0] != T:
        raise ValueError(f"v must have {T} tokens, got {v.shape[0]}")
    Hq = q_step = 0
    if q is not None:
        Hq = q.shape[1] if q.dim() == 3 else 0
        q_step = _rows(q, "q", dt, (Hq, D), index)
        if q.shape[0] != T:
            raise ValueError(f"q must have {T} tokens, got {q.shape[0]}")
        if out is None:
            out = torch.empty((T, Hq, D), dtype=dt, device=dev)
        else:
            _need(out, "out", dt, (T, Hq, D), dev)
    elif out is not None:
        raise ValueError("out is given without q")
    positions = rot = 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    if cos is not None:
        if cos.dim() != 2:
            raise ValueError("cos must be 2-D [positions, rot_dim / 2]")
        positions, half = shape = cos.shape
        rot = 2 * half
        if not (_is(cos, torch.float32, shape, index) and _is(sin, torch.float32, shape, index)):
            _need(cos, "cos", torch.float32, None, dev)
            _need(sin, "sin", torch.float32, shape, dev)
    st = _lib.lib().q8_kv_append(_ptr(q), q_step, k.data_ptr(), k_step, v.data_ptr(), v_step, _DT[dt], T, Hq, Hkv, D,
                                 _ptr(cos), _ptr(sin), positions, rot, interleaved, batch.q_start.data_ptr(),
                                 batch.kv_len.data_ptr(), batch.block_table.data_ptr(), S, max_pages, batch.max_q,
                                 cache.k.data_ptr(), cache.k_exp.data_ptr(), cache.v.data_ptr(),
                                 cache.v_exp.data_ptr(), P, page, _ptr(out), _raw_stream(index))
    if st:
        _lib.check("q8_kv_append", st)
    return out


def q8_attention_workspace_bytes(T: int, heads: int, kv_heads: int, dim: int, seqs: int, max_q: int, max_kv: int,
                                 window: int = 0) -> int:
    return int(_lib.lib().q8_attention_workspace_bytes(T, heads, kv_heads, dim, seqs, max_q, max_kv, window))


def q8_attention_kv8(q: torch.Tensor, cache: KvCache, batch: KvBatch, scale: Optional[float] = None,
                     causal: bool = True, window: int = 0, lse: bool = False,
                     out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Attention of the new queries q [T, heads, dim] (bf16 or fp16, any token
    stride) over the cache; scale defaults to 1/sqrt(dim).  Returns out
    [T, heads, dim] (and the log-sum-exp float32 [T, heads] if lse)."""
    if not lse and workspace is None:
        r = _fast().attention_kv8(q, cache, batch, scale, causal, window, out)
        if r is not NotImplemented:
            return _result("q8_attention_kv8", r)
    index, dev = _cuda_index(q, "q"), q.device
    P, Hkv, page, D, S, max_pages = _check_kv(cache, batch, dev, index)
    dt = q.dtype
    if dt not in (torch.bfloat16, torch.float16):
        raise TypeError("q8_attention_kv8: q must be bfloat16 or float16")
    T, Hq = q.shape[:2] if q.dim() == 3 else (0, 0)
    q_step = _rows(q, "q", dt, (Hq, D), index)
    if out is None:
        y = torch.empty((T, Hq, D), dtype=dt, device=dev)
    else:
        y = out
        _need(y, "out", dt, (T, Hq, D), dev)
    le = torch.empty(T, Hq, dtype=torch.float32, device=dev) if lse else None
    L = _lib.lib()
    max_q, max_kv = batch.max_q, batch.max_kv
    ws = workspace
    if ws is None:
        wsn = L.q8_attention_workspace_bytes(T, Hq, Hkv, D, S, max_q, max_kv, window)
        if wsn:
            ws = torch.empty(wsn, dtype=torch.uint8, device=dev)
    else:
        wsn = ws.nbytes
        if ws.get_device() != index or not ws.is_contiguous():
            _need(ws, "workspace", None, None, dev)
    st = L.q8_attention_kv8(q.data_ptr(), q_step, _DT[dt], T, Hq, Hkv, D, batch.q_start.data_ptr(),
                            batch.kv_len.data_ptr(), batch.block_table.data_ptr(), S, max_pages, max_q, max_kv,
                            cache.k.data_ptr(), cache.k_exp.data_ptr(), cache.v.data_ptr(), cache.v_exp.data_ptr(), P,
                            page, 1.0 / math.sqrt(D) if scale is None else scale, causal, window, y.data_ptr(),
                            _ptr(le), _ptr(ws), wsn, _raw_stream(index))
    if st:
        _lib.check("q8_attention_kv8", st)
    return (y, le) if lse else y


def _need_codes(t: torch.Tensor, name: str, shape=None, dev=None) -> None:
    _need(t, name, None, shape, dev)
    if t.dtype not in _CODES:
        raise TypeError(f"{name} must be uint8 or float8_e4m3fn, got {t.dtype}")


def q8_quantize_weight_block(w: torch.Tensor):
    """FP8 weights with one scale per 128 x 128 block: (wq uint8 e4m3 codes [N, K],
    w_scale float32 [ceil(N/128), ceil(K/128)])."""
    _need(w, "w")
    if w.dim() != 2:
        raise ValueError("w must be 2-D")
    N, K = w.shape
    dev = w.device
    wq = torch.empty(N, K, dtype=torch.uint8, device=dev)
    ws = torch.empty(-(-N // 128), -(-K // 128), dtype=torch.float32, device=dev)
    st = _lib.lib().q8_quantize_weight_block(_ptr(w), _DT[w.dtype], N, K, _ptr(wq), _ptr(ws), _stream(dev))
    _lib.check("q8_quantize_weight_block", st)
    return wq, ws


def q8_quantize_act_block(x: torch.Tensor, out=None):
    """FP8 activations with one scale per token and 128 features: (xq uint8 e4m3
    codes [M, K], x_scale float32 [ceil(K/128), M]); `out` may supply both."""
    _need(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    M, K = x.shape
    dev = x.device
    G = -(-K // 128)
    xq, xs = out if out is not None else (torch.empty(M, K, dtype=torch.uint8, device=dev),
                                          torch.empty(G, M, dtype=torch.float32, device=dev))
    _need(xq, "xq", torch.uint8, (M, K), dev)
    _need(xs, "x_scale", torch.float32, (G, M), dev)
    st = _lib.lib().q8_quantize_act_block(_ptr(x), _DT[x.dtype], M, K, _ptr(xq), _ptr(xs), _stream(dev))
    _lib.check("q8_quantize_act_block", st)
    return xq, xs


def q8_gemm_fp8_block(xq: torch.Tensor, x_scale: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor,
                      bias: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                      out: Optional[torch.Tensor] = None):
    """The block-scaled FP8 product on quantized operands, codes as uint8 or
    float8_e4m3fn (bf16 or fp16 out)."""
    _need_codes(xq, "xq")
    dev = xq.device
    M, K = xq.shape
    N = wq.shape[0]
    G = -(-K // 128)
    _need(x_scale, "x_scale", torch.float32, (G, M), dev)
    _need_codes(wq, "wq", (N, K), dev)
    _need(w_scale, "w_scale", torch.float32, (-(-N // 128), G), dev)
    if bias is not None:
        _need(bias, "bias", torch.float32, (N,), dev)
    y = out if out is not None else torch.empty(M, N, dtype=out_dtype, device=dev)
    _need(y, "y", out_dtype, (M, N), dev)
    st = _lib.lib().q8_gemm_fp8_block(_ptr(xq), _ptr(x_scale), M, K, _ptr(wq), _ptr(w_scale), N, _ptr(bias), _ptr(y),
                                      _DT[out_dtype], _stream(dev))
    _lib.check("q8_gemm_fp8_block", st)
    return y


def q8_linear_fp8_block(x: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor,
                        bias: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                        out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Linear layer with block-scaled FP8 weights (from q8_quantize_weight_block,
    or a checkpoint's float8_e4m3fn codes and scales) and activations quantized per token and 128 features; bf16 or fp16 out
    (default: x's dtype, bf16 for a float32 x)."""
    if workspace is None:
        r = _fast().linear_fp8_block(x, wq, w_scale, bias, out_dtype, out)
        if r is not NotImplemented:
            return _result("q8_linear_fp8_block", r)
    index, dev = _cuda_index(x, "x"), x.device
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    M, K = x.shape
    N = wq.shape[0]
    xd = x.dtype
    blocks = (-(-N // 128), -(-K // 128))
    if not (x.is_contiguous() and wq.dtype in _CODES and _is(wq, wq.dtype, (N, K), index) and _is(w_scale, torch.float32, blocks, index)
            and (bias is None or _is(bias, torch.float32, (N,), index))):
        _need(x, "x")
        _need_codes(wq, "wq", (N, K), dev)
        _need(w_scale, "w_scale", torch.float32, blocks, dev)
        _need(bias, "bias", torch.float32, (N,), dev)
    out_dtype = out_dtype or (torch.bfloat16 if xd is torch.float32 else xd)
    if out is None:
        y = torch.empty((M, N), dtype=out_dtype, device=dev)
    else:
        y = out
        _need(y, "y", out_dtype, (M, N), dev)
    L = _lib.lib()
    ws = workspace
    if ws is None:
        wsn = L.q8_workspace_bytes(_lib.Q8_OP_FP8_BLOCK, M, N, K)
        if wsn:
            ws = torch.empty(wsn, dtype=torch.uint8, device=dev)
    else:
        _need(ws, "workspace", None, None, dev)
        wsn = ws.nbytes
    st = L.q8_linear_fp8_block(x.data_ptr(), _DT[xd], M, K, wq.data_ptr(), w_scale.data_ptr(), N, _ptr(bias),
                               y.data_ptr(), _DT[out_dtype], _ptr(ws), wsn, _raw_stream(index))
    if st:
        _lib.check("q8_linear_fp8_block", st)
    return y


def q8_bench_mfma_loop(fmt: str, iters: int, workgroups: int, sink: torch.Tensor) -> None:
    """Measurement helper (include/q8_bench.h): a register-only MFMA loop,
    fmt "int8_sym" (int8 32x32x32) or "fp8_e4m3" (fp8 32x32x64); sink is a
    device int32 tensor of workgroups * 256 elements."""
    dev = sink.device
    _need(sink, "sink", torch.int32, (workgroups * 256,), dev)
    st = _lib.lib().q8_bench_mfma_loop(_FMT[fmt], iters, workgroups, _ptr(sink), _stream(dev))
    _lib.check("q8_bench_mfma_loop", st)


def q8_probe_fp8_mfma(a: torch.Tensor, b: torch.Tensor, c: torch.Tensor) -> torch.Tensor:
    """Measurement helper (include/q8_bench.h): d = c + a . b^T through one
    FP8 MFMA per problem.  a, b: uint8 e4m3 codes [P, 32, 64]; c: float32
    [P, 32, 32]; returns d float32 [P, 32, 32]."""
    dev = a.device
    P = a.shape[0]
    _need(a, "a", torch.uint8, (P, 32, 64), dev)
    _need(b, "b", torch.uint8, (P, 32, 64), dev)
    _need(c, "c", torch.float32, (P, 32, 32), dev)
    d = torch.empty(P, 32, 32, dtype=torch.float32, device=dev)
    st = _lib.lib().q8_probe_fp8_mfma(_ptr(a), _ptr(b), _ptr(c), _ptr(d), P, _stream(dev))
    _lib.check("q8_probe_fp8_mfma", st)
    return d


def q8_gemm_tile(op: str, M: int, N: int, K: int) -> tuple:
    """Introspection helper (include/q8_bench.h): the (rows, columns) output
    tile of the MFMA GEMM that a call of op ("linear", "static", "decomp",
    "fp8") runs at this shape; (0, 0) where none runs."""
    bm, bn = ctypes.c_int32(0), ctypes.c_int32(0)
    st = _lib.lib().q8_gemm_tile(_OP[op], M, N, K, ctypes.byref(bm), ctypes.byref(bn))
    _lib.check("q8_gemm_tile", st)
    return bm.value, bn.value


def q8_bench_stream_read(src: torch.Tensor, workgroups: int, sink: torch.Tensor) -> None:
    """Measurement helper (include/q8_bench.h): one streaming read of the
    device tensor src (its bytes, a multiple of 16); sink is a device int32
    tensor of workgroups * 256 elements."""
    dev = src.device
    _need(src, "src", None, None, dev)
    _need(sink, "sink", torch.int32, (workgroups * 256,), dev)
    nbytes = src.numel() * src.element_size()
    st = _lib.lib().q8_bench_stream_read(_ptr(src), nbytes, workgroups, _ptr(sink), _stream(dev))
    _lib.check("q8_bench_stream_read", st)
