"""The 8-bit serving path over the libdq C ABI (marshalling only, like `api`): row quantization,
the INT8 product and linear layer, the paged key/value cache and the attention that reads it.

Each helper checks shapes, dtypes and devices, allocates what it is not given (on the input's
device and on the stream that it launches on) and passes raw pointers to the C entry point of
the same name. Calls go to the current stream of the input's device unless `stream` is given;
outputs then belong to that stream until it has been waited for.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .api import DQError, _check, _dtype_code, _need_cuda

# A decode step's kernels take a few microseconds, so the helpers are written for few Python
# operations a call: conditions are tested in line, and what is wrong is worked out only when
# one of them fails; the stream is read as a raw handle, and results are allocated by strides.
_device = torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream
_alloc = torch.empty_strided


def _place(t: torch.Tensor, stream):
    """The context (device, stream) in which a call on `t` allocates and launches."""
    if stream is None:
        return torch.cuda.device(t.device)
    if stream.device != t.device:
        raise ValueError("stream and tensors are on different devices")
    return torch.cuda.stream(stream)               # also makes the stream's device current


def _expect(t, dev: int, name: str, dtype) -> None:
    """A CUDA tensor of the call's device and the given dtype."""
    if not (isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype is dtype):
        _need_cuda(t, name)
        if t.get_device() != dev:
            raise ValueError(name + " is on another device")
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))


def _vector(t, dev: int, name: str, n: int, dtype) -> int:
    """Address of a contiguous vector of n entries."""
    if (isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype is dtype
            and t.shape == (n,) and t.is_contiguous()):
        return t.data_ptr()
    _expect(t, dev, name, dtype)
    raise ValueError("%s must be contiguous with %d entries" % (name, n))


def _scratch(workspace, need: int, like: torch.Tensor) -> torch.Tensor:
    if workspace is None:
        return _alloc((need,), (1,), dtype=torch.uint8, device=like.device)
    _expect(workspace, like.get_device(), "workspace", torch.uint8)
    if not workspace.is_contiguous() or workspace.numel() < need:
        raise ValueError("workspace needs %d contiguous bytes" % need)
    return workspace


# The entry points ask for at least 16 bytes of workspace even where the plan of a call uses
# none; those calls, which neither read nor write them, are given the same 16 bytes.
_UNUSED_BYTES = 16
_unused: dict = {}


def _unused_scratch(like: torch.Tensor) -> int:
    t = _unused.get(like.device)
    if t is None:
        t = _unused[like.device] = torch.empty((_UNUSED_BYTES,), dtype=torch.uint8,
                                               device=like.device)
    return t.data_ptr()


def _rows_of(X: torch.Tensor, name: str):
    """(rows, columns, row pitch) of a 2-D row-major tensor. A single row's stride carries no
    meaning and may be anything."""
    if X.dim() != 2:
        raise ValueError(name + " must be 2-D row-major")
    (T, n), (pitch, one) = X.shape, X.stride()
    if one != 1 and n > 1 and T > 0:
        raise ValueError(name + " must be 2-D row-major")
    return T, n, (pitch if T > 1 else n)


def row_quant(X: torch.Tensor, c: torch.Tensor | None = None, stream=None,
              out: dict | None = None) -> dict:
    """dq_row_quant: INT8 codes of fl32(X * c) with one fp32 scale per row.

    Activations: X [tokens, channels] with the solver's c. Weights: X [out, in] with 1 / c.
    Returns {"codes": int8 [rows, n], "scales": fp32 [rows]} (written into `out` if given)."""
    _need_cuda(X, "X")
    dev = X.get_device()
    if stream is not None or dev != _device():
        with _place(X, stream):
            return row_quant(X, c, None, out)
    T, n, pitch = _rows_of(X, "X")
    dt = _dtype_code(X)
    cp = None if c is None else _vector(c, dev, "c", n, torch.float32)
    if out is None:
        out = {"codes": _alloc((T, n), (n, 1), dtype=torch.int8, device=X.device),
               "scales": _alloc((T,), (1,), dtype=torch.float32, device=X.device)}
        q, s = out["codes"].data_ptr(), out["scales"].data_ptr()
    else:
        rows, cols, q, s = _codes_of(out, dev, "out")
        if rows != T or cols != n:
            raise ValueError("out has another shape than X")
    st = _lib.get().dq_row_quant(X.data_ptr(), dt, T, n, pitch, cp, q, s, _raw_stream(dev))
    if st:
        _check(st, "dq_row_quant")
    return out


def _codes_of(d: dict, dev: int, name: str):
    """(rows, columns, address of the codes, address of the scales)"""
    q = d["codes"]
    _expect(q, dev, name + " codes", torch.int8)
    if q.dim() != 2 or not q.is_contiguous():
        raise ValueError(name + " codes must be 2-D and contiguous")
    T, K = q.shape
    return T, K, q.data_ptr(), _vector(d["scales"], dev, name + " scales", T, torch.float32)


def _result(out, T: int, N: int, dtype, like: torch.Tensor):
    """(tensor, dtype code, row pitch) of a product's result."""
    if dtype is torch.float32:
        code = _lib.DQ_F32
    elif dtype is torch.bfloat16:
        code = _lib.DQ_BF16
    else:
        raise TypeError("out_dtype must be float32 or bfloat16")
    if out is None:
        return _alloc((T, N), (N, 1), dtype=dtype, device=like.device), code, N
    _expect(out, like.get_device(), "out", dtype)
    if tuple(out.shape) != (T, N):
        raise ValueError("out must be [%d, %d]" % (T, N))
    return out, code, _rows_of(out, "out")[2]


def w8a8_gemm(x: dict, w: dict, out_dtype=torch.float32, stream=None,
              workspace: torch.Tensor | None = None,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """dq_w8a8_gemm: y[T, N] from two row_quant results, x (tokens) and w (output channels)."""
    xt = x["codes"]
    _need_cuda(xt, "x codes")
    dev = xt.get_device()
    if stream is not None or dev != _device():
        with _place(xt, stream):
            return w8a8_gemm(x, w, out_dtype, None, workspace, out)
    T, K, xq, xs = _codes_of(x, dev, "x")
    N, Kw, wq, ws = _codes_of(w, dev, "w")
    if Kw != K:
        raise ValueError("activation and weight K differ")
    lib = _lib.get()
    need = lib.dq_w8a8_gemm_workspace_bytes(T, N, K)
    if need == 0:
        raise DQError(_lib.DQ_ERR_SHAPE, "K must be a multiple of 16 up to 131072")
    y, code, pitch = _result(out, T, N, out_dtype, xt)
    if workspace is None and need <= _UNUSED_BYTES:
        sp = _unused_scratch(xt)
    else:
        workspace = _scratch(workspace, need, xt)
        sp = workspace.data_ptr()
    st = lib.dq_w8a8_gemm(xq, xs, T, wq, ws, N, K, y.data_ptr(), code, pitch, sp, need,
                          _raw_stream(dev))
    if st:
        _check(st, "dq_w8a8_gemm")
    return y


def w8a8_linear(X: torch.Tensor, w: dict, c: torch.Tensor | None = None,
                out_dtype=torch.bfloat16, stream=None, workspace: torch.Tensor | None = None,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """dq_w8a8_linear: y[T, N] = row_quant(X, c) times an 8-bit weight `w`."""
    _need_cuda(X, "X")
    dev = X.get_device()
    if stream is not None or dev != _device():
        with _place(X, stream):
            return w8a8_linear(X, w, c, out_dtype, None, workspace, out)
    T, K, pitch = _rows_of(X, "X")
    dt = _dtype_code(X)
    N, Kw, wq, ws = _codes_of(w, dev, "w")
    if Kw != K:
        raise ValueError("activation and weight K differ")
    cp = None if c is None else _vector(c, dev, "c", K, torch.float32)
    lib = _lib.get()
    need = lib.dq_w8a8_linear_workspace_bytes(T, N, K)
    if need == 0:
        raise DQError(_lib.DQ_ERR_SHAPE, "K must be a multiple of 16 up to 131072")
    y, code, ypitch = _result(out, T, N, out_dtype, X)
    sp = _scratch(workspace, need, X)
    st = lib.dq_w8a8_linear(X.data_ptr(), dt, T, K, pitch, cp, wq, ws, N, y.data_ptr(), code,
                            ypitch, sp.data_ptr(), sp.numel(), _raw_stream(dev))
    if st:
        _check(st, "dq_w8a8_linear")
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


def _cache_of(cache: dict, dev: int) -> _lib.dq_kv_cache:
    k, v = cache["k"], cache["v"]
    _need_cuda(k, "cache k")
    dtype = k.dtype
    shape, strides = k.shape, k.stride()
    if dtype is torch.int8:
        kind = _lib.DQ_CACHE_INT8
    elif dtype is torch.bfloat16:
        kind = _lib.DQ_CACHE_BF16
    else:
        raise TypeError("the cache must be bfloat16 or int8, got %s" % dtype)
    if k.get_device() != dev:
        _expect(k, dev, "cache k", dtype)
    _expect(v, dev, "cache v", dtype)
    if len(shape) != 4 or v.shape != shape or v.stride() != strides or strides[3] != 1:
        raise ValueError("cache k and v must be [pages, kv_heads, page_size, head_dim] with the "
                         "same strides and contiguous channels")
    P, G, S, D = shape
    ps, hs, rs, _ = strides
    # the stride of an axis of one entry carries no meaning
    if P == 1:
        ps = G * S * D
    if G == 1:
        hs = S * D
    if kind == _lib.DQ_CACHE_BF16:
        return _lib.dq_kv_cache(kind, S, D, G, P, k.data_ptr(), v.data_ptr(), ps, hs, rs, None,
                                None)
    ks, vs = cache["k_scales"], cache["v_scales"]
    _expect(ks, dev, "cache k_scales", torch.float32)
    _expect(vs, dev, "cache v_scales", torch.float32)
    rows = (P, G, S)
    if ks.shape != rows or vs.shape != rows or not (ks.is_contiguous() and vs.is_contiguous()):
        raise ValueError("cache scales must be contiguous [pages, kv_heads, page_size]")
    return _lib.dq_kv_cache(kind, S, D, G, P, k.data_ptr(), v.data_ptr(), ps, hs, rs,
                            ks.data_ptr(), vs.data_ptr())


def _heads(x: torch.Tensor, dev: int, name: str, dtype, T: int, H: int, D: int) -> int:
    """Token stride of [T, H, D] of the call's device and dtype with contiguous heads."""
    if (isinstance(x, torch.Tensor) and x.get_device() == dev and x.dtype is dtype
            and x.shape == (T, H, D)):
        t, h, d = x.stride()
        if (d == 1 and (h == D or H == 1)) or T == 0:
            return t if T > 1 else H * D
        raise ValueError("%s must have contiguous heads and channels" % name)
    _expect(x, dev, name, dtype)
    raise ValueError("%s must be [%d, %d, %d]" % (name, T, H, D))


def kv_append(k: torch.Tensor, v: torch.Tensor, cache: dict, slots: torch.Tensor,
              positions: torch.Tensor | None = None, cos: torch.Tensor | None = None,
              sin: torch.Tensor | None = None, q: torch.Tensor | None = None,
              interleaved: bool = False, q_out: torch.Tensor | None = None, stream=None):
    """dq_kv_append: keys and values [T, kv_heads, head_dim] into the cache's `slots` (int64,
    page * page_size + row; negative: not stored), the keys rotated by `positions` (int32) into
    cos, sin [rows, dim / 2] (fp32) where these are given. With q [T, heads, head_dim], returns
    the rotated queries in bfloat16 (in `q_out` if given, which may be q)."""
    _need_cuda(k, "k")
    dev = k.get_device()
    if stream is not None or dev != _device():
        with _place(k, stream):
            return kv_append(k, v, cache, slots, positions, cos, sin, q, interleaved, q_out)
    dtype = k.dtype
    dt = _dtype_code(k)
    c = _cache_of(cache, dev)
    T, D, G = k.shape[0] if k.dim() else 0, c.head_dim, c.kv_heads
    ks = _heads(k, dev, "k", dtype, T, G, D)
    vs = _heads(v, dev, "v", dtype, T, G, D)
    sp = _vector(slots, dev, "slots", T, torch.int64)
    rot = None
    if positions is not None or cos is not None or sin is not None:
        if positions is None or cos is None or sin is None:
            raise ValueError("positions, cos and sin go together")
        pp = _vector(positions, dev, "positions", T, torch.int32)
        _expect(cos, dev, "cos", torch.float32)
        _expect(sin, dev, "sin", torch.float32)
        shape = cos.shape
        if len(shape) != 2 or sin.shape != shape or not (cos.is_contiguous()
                                                         and sin.is_contiguous()):
            raise ValueError("cos and sin must be contiguous [rows, dim / 2]")
        rows, half = shape
        rot = ctypes.byref(_lib.dq_rotary(cos.data_ptr(), sin.data_ptr(), pp, rows, 2 * half,
                                          1 if interleaved else 0))
    qp = op = None
    H = qs = os = 0
    if q is not None:
        H = q.shape[1] if q.dim() == 3 else 0
        qs = _heads(q, dev, "q", dtype, T, H, D)
        if q_out is None:
            os = H * D
            q_out = _alloc((T, H, D), (os, D, 1), dtype=torch.bfloat16, device=k.device)
        else:
            os = _heads(q_out, dev, "q_out", torch.bfloat16, T, H, D)
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    st = _lib.get().dq_kv_append(ctypes.byref(c), T, dt, k.data_ptr(), ks, v.data_ptr(), vs, sp,
                                 rot, qp, qs, H, op, os, _raw_stream(dev))
    if st:
        _check(st, "dq_kv_append")
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
    dev = q.get_device()
    if stream is not None or dev != _device():
        with _place(q, stream):
            return paged_attention(q, cache, page_table, lengths, q_starts, max_q, max_len,
                                   causal, scale, out, None, workspace)
    c = _cache_of(cache, dev)
    T, H, D = (*q.shape[:2], c.head_dim) if q.dim() == 3 else (0, 0, c.head_dim)
    qs = _heads(q, dev, "q", torch.bfloat16, T, H, D)
    _expect(page_table, dev, "page_table", torch.int32)
    if page_table.dim() != 2:
        raise ValueError("page_table must be 2-D row-major")
    B, width = page_table.shape
    pitch, one = page_table.stride()
    if one != 1 and width > 1 and B > 0:
        raise ValueError("page_table must be 2-D row-major")
    if B <= 1:
        pitch = width
    lp = _vector(lengths, dev, "lengths", B, torch.int32)
    sp = None
    if q_starts is not None:
        sp = _vector(q_starts, dev, "q_starts", B + 1, torch.int32)
    elif T != B:
        raise ValueError("without q_starts there is one token per sequence")
    if max_q is None:
        max_q = T if sp is not None else 1
    if max_q > T:
        max_q = T
    if max_len is None:
        max_len = width * c.page_size
    elif max_len > width * c.page_size:
        raise ValueError("max_len is more than the page table's width holds")
    if out is None:
        os = H * D
        out = _alloc((T, H, D), (os, D, 1), dtype=torch.bfloat16, device=q.device)
    else:
        os = _heads(out, dev, "out", torch.bfloat16, T, H, D)
    a = _lib.dq_attention(q.data_ptr(), out.data_ptr(), qs, os, T, B, H, 1 if causal else 0, sp,
                          lp, page_table.data_ptr(), pitch, max_q, max_len,
                          D ** -0.5 if scale is None else scale)
    call = _lib.get().dq_paged_attention
    cr, ar = ctypes.byref(c), ctypes.byref(a)
    st = _lib.DQ_ERR_WORKSPACE
    if workspace is None:
        st = call(cr, ar, _unused_scratch(q), _UNUSED_BYTES, _raw_stream(dev))
    if st == _lib.DQ_ERR_WORKSPACE:                # split sequences need room for their parts
        need = _lib.get().dq_paged_attention_workspace_bytes(cr, ar)
        workspace = _scratch(workspace, need, q)
        st = call(cr, ar, workspace.data_ptr(), workspace.numel(), _raw_stream(dev))
    if st:
        _check(st, "dq_paged_attention")
    return out
