"""The 8-bit serving path over the libdq C ABI (marshalling only, like `api`): row quantization,
the INT8 product and linear layer, the paged key/value cache and the attention that reads it.

Each helper checks shapes, dtypes and devices, allocates what it is not given (on the input's
device and on the stream that it launches on) and passes raw pointers to the C entry point of
the same name. Calls go to the current stream of the input's device unless `stream` is given;
outputs then belong to that stream until it has been waited for.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _lib
from .api import DQError, _check, _dtype_code, _need_cuda

_NULL = contextlib.nullcontext()


def _place(t: torch.Tensor, stream):
    """The context (device, stream) in which a call on `t` allocates and launches."""
    if stream is not None:
        if stream.device != t.device:
            raise ValueError("stream and tensors are on different devices")
        return torch.cuda.stream(stream)           # also makes the stream's device current
    if t.device.index != torch.cuda.current_device():
        return torch.cuda.device(t.device)
    return _NULL


def _cur(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _same(t, like: torch.Tensor, name: str, dtype) -> None:
    _need_cuda(t, name)
    if t.device != like.device:
        raise ValueError(name + " is on another device")
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))


def _vector(t, like: torch.Tensor, name: str, n: int, dtype) -> None:
    _same(t, like, name, dtype)
    if t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must be contiguous with %d entries" % (name, n))


def _scratch(workspace, need: int, like: torch.Tensor) -> torch.Tensor:
    if workspace is None:
        return torch.empty((need,), dtype=torch.uint8, device=like.device)
    _same(workspace, like, "workspace", torch.uint8)
    if not workspace.is_contiguous() or workspace.numel() < need:
        raise ValueError("workspace needs %d contiguous bytes" % need)
    return workspace


def _rows_of(X: torch.Tensor, name: str) -> None:
    _need_cuda(X, name)
    if X.dim() != 2 or (X.stride(1) != 1 and X.numel() > 0):
        raise ValueError(name + " must be 2-D row-major")


def _pitch(t: torch.Tensor) -> int:
    # (a single row's stride carries no meaning and may be anything)
    return max(t.stride(0), t.shape[1]) if t.shape[0] > 1 else t.shape[1]


def row_quant(X: torch.Tensor, c: torch.Tensor | None = None, stream=None,
              out: dict | None = None) -> dict:
    """dq_row_quant: INT8 codes of fl32(X * c) with one fp32 scale per row.

    Activations: X [tokens, channels] with the solver's c. Weights: X [out, in] with 1 / c.
    Returns {"codes": int8 [rows, n], "scales": fp32 [rows]} (written into `out` if given)."""
    _rows_of(X, "X")
    dt = _dtype_code(X)
    T, n = X.shape
    if c is not None:
        _vector(c, X, "c", n, torch.float32)
    with _place(X, stream):
        if out is None:
            out = dict(codes=torch.empty((T, n), dtype=torch.int8, device=X.device),
                       scales=torch.empty((T,), dtype=torch.float32, device=X.device))
        else:
            _codes_of(out, X, "out")
            if tuple(out["codes"].shape) != (T, n):
                raise ValueError("out has another shape than X")
        _check(_lib.get().dq_row_quant(X.data_ptr(), dt, T, n, _pitch(X),
                                       None if c is None else c.data_ptr(),
                                       out["codes"].data_ptr(), out["scales"].data_ptr(),
                                       _cur(X)), "dq_row_quant")
    return out


def _codes_of(d: dict, like: torch.Tensor, name: str):
    q, s = d["codes"], d["scales"]
    _same(q, like, name + " codes", torch.int8)
    if q.dim() != 2 or not q.is_contiguous():
        raise ValueError(name + " codes must be 2-D and contiguous")
    _vector(s, like, name + " scales", q.shape[0], torch.float32)
    return q, s


def _result(out, T: int, N: int, dtype, like: torch.Tensor) -> torch.Tensor:
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out_dtype must be float32 or bfloat16")
    if out is None:
        return torch.empty((T, N), dtype=dtype, device=like.device)
    _same(out, like, "out", dtype)
    if tuple(out.shape) != (T, N) or (out.stride(1) != 1 and N > 1):
        raise ValueError("out must be [%d, %d], row-major" % (T, N))
    return out


def w8a8_gemm(x: dict, w: dict, out_dtype=torch.float32, stream=None,
              workspace: torch.Tensor | None = None,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """dq_w8a8_gemm: y[T, N] from two row_quant results, x (tokens) and w (output channels)."""
    xq = x["codes"]
    _need_cuda(xq, "x codes")
    xq, xs = _codes_of(x, xq, "x")
    wq, ws = _codes_of(w, xq, "w")
    T, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] != K:
        raise ValueError("activation and weight K differ")
    lib = _lib.get()
    need = lib.dq_w8a8_gemm_workspace_bytes(T, N, K)
    if need == 0:
        raise DQError(_lib.DQ_ERR_SHAPE, "K must be a multiple of 16 up to 131072")
    with _place(xq, stream):
        y = _result(out, T, N, out_dtype, xq)
        sp = _scratch(workspace, need, xq)
        _check(lib.dq_w8a8_gemm(xq.data_ptr(), xs.data_ptr(), T, wq.data_ptr(), ws.data_ptr(),
                                N, K, y.data_ptr(), _dtype_code(y), _pitch(y), sp.data_ptr(),
                                sp.numel(), _cur(xq)), "dq_w8a8_gemm")
    return y


def w8a8_linear(X: torch.Tensor, w: dict, c: torch.Tensor | None = None,
                out_dtype=torch.bfloat16, stream=None, workspace: torch.Tensor | None = None,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """dq_w8a8_linear: y[T, N] = row_quant(X, c) times an 8-bit weight `w`."""
    _rows_of(X, "X")
    dt = _dtype_code(X)
    wq, ws = _codes_of(w, X, "w")
    T, K = X.shape
    N = wq.shape[0]
    if wq.shape[1] != K:
        raise ValueError("activation and weight K differ")
    if c is not None:
        _vector(c, X, "c", K, torch.float32)
    lib = _lib.get()
    need = lib.dq_w8a8_linear_workspace_bytes(T, N, K)
    if need == 0:
        raise DQError(_lib.DQ_ERR_SHAPE, "K must be a multiple of 16 up to 131072")
    with _place(X, stream):
        y = _result(out, T, N, out_dtype, X)
        sp = _scratch(workspace, need, X)
        _check(lib.dq_w8a8_linear(X.data_ptr(), dt, T, K, _pitch(X),
                                  None if c is None else c.data_ptr(), wq.data_ptr(),
                                  ws.data_ptr(), N, y.data_ptr(), _dtype_code(y), _pitch(y),
                                  sp.data_ptr(), sp.numel(), _cur(X)), "dq_w8a8_linear")
    return y


# ----------------------------------------------------------------------------- paged cache
CACHE_TYPES = {torch.bfloat16: _lib.DQ_CACHE_BF16, torch.int8: _lib.DQ_CACHE_INT8}


def kv_cache(pages: int, kv_heads: int, page_size: int, head_dim: int, dtype=torch.bfloat16,
             device="cuda") -> dict:
    """An empty paged cache: k, v [pages, kv_heads, page_size, head_dim] of bfloat16, or int8
    with k_scales, v_scales [pages, kv_heads, page_size]. Any dict of tensors of these shapes
    with contiguous channels will do, for instance a permuted view of a cache kept token by
    token (k and v with the same strides, the scales contiguous)."""
    if dtype not in CACHE_TYPES:
        raise TypeError("a cache holds bfloat16 or int8")
    shape = (pages, kv_heads, page_size, head_dim)
    d = dict(k=torch.zeros(shape, dtype=dtype, device=device),
             v=torch.zeros(shape, dtype=dtype, device=device))
    if dtype == torch.int8:
        d["k_scales"] = torch.zeros(shape[:3], dtype=torch.float32, device=device)
        d["v_scales"] = torch.zeros(shape[:3], dtype=torch.float32, device=device)
    return d


def _cache_of(cache: dict, like: torch.Tensor) -> _lib.dq_kv_cache:
    k, v = cache["k"], cache["v"]
    if k.dtype not in CACHE_TYPES:
        raise TypeError("the cache must be bfloat16 or int8, got %s" % k.dtype)
    _same(k, like, "cache k", k.dtype)
    _same(v, like, "cache v", k.dtype)
    if k.dim() != 4 or v.shape != k.shape or v.stride() != k.stride() or k.stride(3) != 1:
        raise ValueError("cache k and v must be [pages, kv_heads, page_size, head_dim] with the "
                         "same strides and contiguous channels")
    P, G, S, D = k.shape
    # (the stride of an axis of one entry carries no meaning)
    ps, hs, rs = (s if n > 1 else S * G * D for s, n in zip(k.stride()[:3], (P, G, S)))
    scales = (None, None)
    if k.dtype == torch.int8:
        for name in ("k_scales", "v_scales"):
            _same(cache[name], like, "cache " + name, torch.float32)
            if tuple(cache[name].shape) != (P, G, S) or not cache[name].is_contiguous():
                raise ValueError("cache %s must be contiguous [pages, kv_heads, page_size]" % name)
        scales = (cache["k_scales"].data_ptr(), cache["v_scales"].data_ptr())
    return _lib.dq_kv_cache(CACHE_TYPES[k.dtype], S, D, G, P, k.data_ptr(), v.data_ptr(), ps, hs,
                            rs, *scales)


def _heads(x: torch.Tensor, name: str, T: int, D: int) -> int:
    """Token stride of [T, heads, D] with contiguous heads."""
    if x.dim() != 3 or x.shape[0] != T or x.shape[2] != D:
        raise ValueError("%s must be [%d, heads, %d]" % (name, T, D))
    if x.numel() and (x.stride(2) != 1 or (x.shape[1] > 1 and x.stride(1) != D)):
        raise ValueError("%s must have contiguous heads and channels" % name)
    return x.stride(0) if T > 1 else x.shape[1] * D


def kv_append(k: torch.Tensor, v: torch.Tensor, cache: dict, slots: torch.Tensor,
              positions: torch.Tensor | None = None, cos: torch.Tensor | None = None,
              sin: torch.Tensor | None = None, q: torch.Tensor | None = None,
              interleaved: bool = False, q_out: torch.Tensor | None = None, stream=None):
    """dq_kv_append: keys and values [T, kv_heads, head_dim] into the cache's `slots` (int64,
    page * page_size + row; negative: not stored), the keys rotated by `positions` (int32) into
    cos, sin [rows, dim / 2] (fp32) where these are given. With q [T, heads, head_dim], returns
    the rotated queries in bfloat16 (in `q_out` if given, which may be q)."""
    _need_cuda(k, "k")
    dt = _dtype_code(k)
    _same(v, k, "v", k.dtype)
    c = _cache_of(cache, k)
    T, D, G = k.shape[0], c.head_dim, c.kv_heads
    ks, vs = _heads(k, "k", T, D), _heads(v, "v", T, D)
    if k.dim() != 3 or k.shape[1] != G or v.shape[1] != G:
        raise ValueError("k and v must have the cache's %d heads" % G)
    _vector(slots, k, "slots", T, torch.int64)
    rot = None
    if positions is not None or cos is not None or sin is not None:
        if positions is None or cos is None or sin is None:
            raise ValueError("positions, cos and sin go together")
        _vector(positions, k, "positions", T, torch.int32)
        for t, name in ((cos, "cos"), (sin, "sin")):
            _same(t, k, name, torch.float32)
            if t.dim() != 2 or not t.is_contiguous() or t.shape != cos.shape:
                raise ValueError("cos and sin must be contiguous [rows, dim / 2]")
        rot = _lib.dq_rotary(cos.data_ptr(), sin.data_ptr(), positions.data_ptr(), cos.shape[0],
                             2 * cos.shape[1], int(bool(interleaved)))
    with _place(k, stream):
        qa = (None, 0, 0, None, 0)
        if q is not None:
            _same(q, k, "q", k.dtype)
            qs, H = _heads(q, "q", T, D), q.shape[1]
            if q_out is None:
                q_out = torch.empty((T, H, D), dtype=torch.bfloat16, device=k.device)
            _same(q_out, k, "q_out", torch.bfloat16)
            if q_out.shape != q.shape:
                raise ValueError("q_out must have q's shape")
            qa = (q.data_ptr(), qs, H, q_out.data_ptr(), _heads(q_out, "q_out", T, D))
        elif q_out is not None:
            raise ValueError("q_out without q")
        _check(_lib.get().dq_kv_append(
            ctypes.byref(c), T, dt, k.data_ptr(), ks, v.data_ptr(), vs, slots.data_ptr(),
            None if rot is None else ctypes.byref(rot), *qa, _cur(k)), "dq_kv_append")
    return q_out


def paged_attention(q: torch.Tensor, cache: dict, page_table: torch.Tensor,
                    lengths: torch.Tensor, q_starts: torch.Tensor | None = None,
                    max_q: int | None = None, max_len: int | None = None, causal: bool = True,
                    scale: float | None = None, out: torch.Tensor | None = None, stream=None,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """dq_paged_attention: q [T, heads, head_dim] (bfloat16), the last q_starts[b+1] -
    q_starts[b] tokens of each sequence b of lengths[b] cache rows; without q_starts one token per
    sequence. page_table [sequences, width], lengths and q_starts are int32. max_q and max_len
    bound the new tokens and the rows of one sequence (default: all of q, and the table's
    width): tight bounds make the launch plan fit. Rows of `out` that belong to no sequence are
    left as they are."""
    _need_cuda(q, "q")
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be bfloat16, got %s" % q.dtype)
    c = _cache_of(cache, q)
    if q.dim() != 3:
        raise ValueError("q must be [tokens, heads, head_dim]")
    T, H, D = q.shape[0], q.shape[1], c.head_dim
    qs = _heads(q, "q", T, D)
    _same(page_table, q, "page_table", torch.int32)
    if page_table.dim() != 2 or (page_table.numel() and page_table.stride(1) != 1
                                 and page_table.shape[1] > 1):
        raise ValueError("page_table must be 2-D row-major")
    B, width = page_table.shape
    _vector(lengths, q, "lengths", B, torch.int32)
    if q_starts is not None:
        _vector(q_starts, q, "q_starts", B + 1, torch.int32)
    elif T != B:
        raise ValueError("without q_starts there is one token per sequence")
    if max_q is None:
        max_q = T if q_starts is not None else min(T, 1)
    if max_len is None:
        max_len = width * c.page_size
    elif max_len > width * c.page_size:
        raise ValueError("max_len is more than the page table's width holds")
    with _place(q, stream):
        if out is None:
            out = torch.empty((T, H, D), dtype=torch.bfloat16, device=q.device)
        else:
            _same(out, q, "out", torch.bfloat16)
            if out.shape != q.shape:
                raise ValueError("out must have q's shape")
        a = _lib.dq_attention(q.data_ptr(), out.data_ptr(), qs, _heads(out, "out", T, D), T, B, H,
                              int(bool(causal)), None if q_starts is None else q_starts.data_ptr(),
                              lengths.data_ptr(), page_table.data_ptr(),
                              page_table.stride(0) if B > 1 else width, min(max_q, T), max_len,
                              D ** -0.5 if scale is None else scale)
        lib = _lib.get()
        need = lib.dq_paged_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(a))
        sp = _scratch(workspace, max(need, 16), q)
        _check(lib.dq_paged_attention(ctypes.byref(c), ctypes.byref(a), sp.data_ptr(), sp.numel(),
                                      _cur(q)), "dq_paged_attention")
    return out
