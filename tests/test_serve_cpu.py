"""The 8-bit serving path without a GPU: the entry points refuse bad calls before any CUDA
call, the helpers refuse bad tensors, and the oracle agrees with hand-worked values."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import serve as O

INVALID, SHAPE, DTYPE, WORKSPACE, UNSUPPORTED = 1, 2, 3, 4, 8


@pytest.fixture(scope="module")
def dq():
    from calibration_free_dual_b200 import build
    build.build()
    import calibration_free_dual_b200 as pkg
    return pkg


P = 1 << 20        # a 16-byte aligned address that is never read


def test_row_quant_refusals(dq):
    def call(X=P, dt=1, rows=4, n=64, ldx=64, c=None, q=P, s=P):
        return dq.dq_row_quant(X, dt, rows, n, ldx, c, q, s, None)
    assert call(dt=7) == DTYPE
    assert call(n=24, ldx=24) == SHAPE
    assert call(rows=-1) == INVALID
    assert call(ldx=32) == INVALID
    assert call(ldx=68) == INVALID              # row pitch not a multiple of 16 bytes
    assert call(X=None) == INVALID
    assert call(X=P + 2) == INVALID
    assert call(c=P + 4) == INVALID
    assert call(q=P + 8) == INVALID
    assert call(s=None) == INVALID
    assert call(rows=0, X=None, q=None, s=None) == 0


def test_w8a8_refusals(dq):
    def gemm(x=P, xs=P, T=4, w=P, ws=P, N=8, K=64, y=P, dt=0, ldy=8, sp=P, nb=1 << 30):
        return dq.dq_w8a8_gemm(x, xs, T, w, ws, N, K, y, dt, ldy, sp, nb, None)
    assert gemm(dt=9) == DTYPE
    assert gemm(K=72) == SHAPE
    assert gemm(K=131072 + 16) == SHAPE         # the int32 sum could overflow
    assert gemm(T=-1) == INVALID
    assert gemm(ldy=7) == INVALID
    for name in ("x", "xs", "w", "ws", "y"):
        assert gemm(**{name: None}) == INVALID
    assert gemm(x=P + 8) == INVALID
    assert gemm(w=P + 4) == INVALID
    assert gemm(sp=None) == WORKSPACE
    assert gemm(nb=0) == WORKSPACE
    assert gemm(T=0, x=None) == 0
    assert dq.dq_w8a8_gemm_workspace_bytes(4, 8, 72) == 0
    assert dq.dq_w8a8_linear_workspace_bytes(4, 8, 131088) == 0
    assert dq.dq_w8a8_linear_workspace_bytes(33, 8, 64) > 33 * 64

    def lin(X=P, dt=1, T=4, K=64, ldx=64, c=None, w=P, ws=P, N=8, y=P, ydt=1, ldy=8, sp=P,
            nb=1 << 30):
        return dq.dq_w8a8_linear(X, dt, T, K, ldx, c, w, ws, N, y, ydt, ldy, sp, nb, None)
    assert lin(dt=3) == DTYPE
    assert lin(ydt=3) == DTYPE
    assert lin(ldx=48) == INVALID
    assert lin(X=P + 8) == INVALID
    assert lin(sp=P + 8) == INVALID
    assert lin(nb=100) == WORKSPACE
    assert lin(T=0, X=None) == 0


def _cache(dq, **kw):
    d = dict(kind=0, page_size=16, head_dim=64, kv_heads=2, pages=4, k=P, v=P,
             page_stride=2 * 16 * 64, head_stride=16 * 64, row_stride=64, k_scales=P, v_scales=P)
    d.update(kw)
    return dq.dq_kv_cache(*[d[n] for n, _ in dq.dq_kv_cache._fields_])


BAD_CACHES = [(dict(kind=2), DTYPE), (dict(page_size=24), UNSUPPORTED),
              (dict(head_dim=96), UNSUPPORTED), (dict(kv_heads=0), INVALID),
              (dict(pages=0), INVALID), (dict(k=None), INVALID), (dict(v=P + 8), INVALID),
              (dict(row_stride=60), INVALID), (dict(row_stride=68), INVALID),
              (dict(head_stride=1028), INVALID), (dict(page_stride=0), INVALID),
              (dict(kind=1, k_scales=None), INVALID), (dict(kind=1, head_stride=1032), INVALID)]


@pytest.mark.parametrize("bad,want", BAD_CACHES)
def test_append_and_attention_refuse_bad_caches(dq, bad, want):
    c = _cache(dq, **bad)
    r = dq.dq_kv_append(ctypes.byref(c), 1, 1, P, 128, P, 128, P, None, None, 0, 0, None, 0, None)
    assert r == want
    a = _attn(dq)
    assert dq.dq_paged_attention(ctypes.byref(c), ctypes.byref(a), P, 1 << 30, None) == want


def test_append_refusals(dq):
    c = _cache(dq)

    def call(T=3, dt=1, k=P, ks=128, v=P, vs=128, slots=P, rot=None, q=None, qs=0, H=0, qo=None,
             qos=0, cache=ctypes.byref(c)):
        r = None if rot is None else ctypes.byref(dq.dq_rotary(*rot))
        return dq.dq_kv_append(cache, T, dt, k, ks, v, vs, slots, r, q, qs, H, qo, qos, None)
    assert call(cache=None) == INVALID
    assert call(dt=5) == DTYPE
    assert call(T=-1) == INVALID
    assert call(ks=64) == INVALID
    assert call(vs=132) == INVALID
    assert call(k=None) == INVALID
    assert call(slots=None) == INVALID
    assert call(slots=P + 4) == INVALID
    good = (P, P, P, 100, 64, 0)
    assert call(rot=good[:4] + (12, 0)) == SHAPE
    assert call(rot=good[:4] + (72, 0)) == SHAPE
    assert call(rot=(P, P, P, 0, 64, 0)) == INVALID
    assert call(rot=(None, P, P, 100, 64, 0)) == INVALID
    assert call(rot=(P, P + 4, P, 100, 64, 0)) == INVALID
    assert call(q=P, qs=256, H=4, qo=None, qos=256) == INVALID
    assert call(q=P, qs=128, H=4, qo=P * 2, qos=256) == INVALID
    assert call(q=P, qs=256, H=4, qo=P, qos=264) == INVALID          # in place, another stride
    assert call(dt=0, q=P, qs=256, H=4, qo=P, qos=256) == INVALID    # in place, another type
    assert call(T=0, k=None, v=None, slots=None) == 0


def _attn(dq, **kw):
    d = dict(q=P, out=P, q_stride=256, out_stride=256, tokens=3, sequences=2, heads=4, causal=1,
             q_starts=P, lengths=P, page_table=P, table_stride=4, max_q=2, max_len=64, scale=0.125)
    d.update(kw)
    return dq.dq_attention(*[d[n] for n, _ in dq.dq_attention._fields_])


def test_attention_refusals(dq):
    c = _cache(dq)

    def call(sp=P, nb=1 << 40, **kw):
        return dq.dq_paged_attention(ctypes.byref(c), ctypes.byref(_attn(dq, **kw)), sp, nb, None)
    assert dq.dq_paged_attention(ctypes.byref(c), None, P, 1 << 30, None) == INVALID
    assert call(heads=3) == SHAPE
    assert call(heads=2 * 129, q_stride=2 * 129 * 64, out_stride=2 * 129 * 64) == UNSUPPORTED
    assert call(tokens=-1) == INVALID
    assert call(max_q=4) == SHAPE
    assert call(sequences=65536) == SHAPE
    assert call(q_stride=192) == INVALID
    assert call(out_stride=260) == INVALID
    assert call(scale=float("inf")) == INVALID
    assert call(q_starts=None) == INVALID                 # 3 tokens, 2 sequences
    assert call(table_stride=3) == INVALID                # 64 rows need 4 pages
    for name in ("q", "out", "lengths", "page_table"):
        assert call(**{name: None}) == INVALID
    assert call(q=P + 8) == INVALID
    assert call(sp=None) == WORKSPACE
    assert call(sp=P + 4) == INVALID
    assert call(tokens=0, max_q=0, q=None) == 0
    assert call(sequences=0) == 0
    need = dq.dq_paged_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(
        _attn(dq, max_len=100000, table_stride=6250)))
    assert need > 16
    assert call(nb=need - 1, max_len=100000, table_stride=6250) == WORKSPACE
    bad = _attn(dq, heads=3)
    assert dq.dq_paged_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(bad)) == 0


def test_helpers_refuse_cpu_tensors(dq):
    x = torch.zeros(4, 64)
    w = dict(codes=torch.zeros(8, 64, dtype=torch.int8), scales=torch.zeros(8))
    with pytest.raises(TypeError):
        dq.row_quant(x)
    with pytest.raises(TypeError):
        dq.w8a8_linear(x, w)
    with pytest.raises(TypeError):
        dq.w8a8_gemm(w, w)
    cache = dq.kv_cache(4, 2, 16, 64, device="cpu")
    kv = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        dq.kv_append(kv, kv, cache, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError):
        dq.paged_attention(torch.zeros(1, 4, 64, dtype=torch.bfloat16), cache,
                           torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        dq.kv_cache(4, 2, 16, 64, dtype=torch.float16, device="cpu")


def test_oracle_row_quant_by_hand():
    q, d = O.row_quant(np.array([[1.0, -127.0, 63.5, 0.25], [0.0, 0.0, 0.0, 0.0],
                                 [2.0 ** -140, 0.0, 0.0, -2.0 ** -139]]))
    assert d.tolist() == [1.0, 0.0, 2.0 ** -126]
    # 63.5 is a tie: to even
    assert q.tolist() == [[1, -127, 64, 0], [0, 0, 0, 0], [0, 0, 0, 0]]


def test_oracle_attention_by_hand():
    # equal scores: the mean of the visible values
    q = np.zeros((2, 1, 64))
    k = np.ones((3, 1, 64))
    v = np.arange(3.0)[:, None, None] * np.ones((3, 1, 64))
    o, _, _ = O.attention(q, k, v, True, 1.0)
    assert np.allclose(o[0], 0.5) and np.allclose(o[1], 1.0)
    o, _, _ = O.attention(np.zeros((5, 1, 64)), k, v, True, 1.0)
    assert np.all(o[:2] == 0) and np.all(o[2] == 0) and np.allclose(o[4], 1.0)


def test_oracle_rotation_by_hand():
    c, s = np.array([[1.0, 0.0]]), np.array([[0.0, 1.0]])
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    assert O.rotate(x, c, s, [0]).tolist() == [[[1.0, -4.0, 3.0, 2.0, 5.0]]]
    assert O.rotate(x, c, s, [0], True).tolist() == [[[1.0, 2.0, -4.0, 3.0, 5.0]]]
