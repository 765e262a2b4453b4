"""The 8-bit serving path on the GPU against the oracle's plain definitions in 64 bits.

Codes, scales, the INT8 product and the rotated, quantized cache rows are defined down to single
binary32 operations, so they agree bit for bit (bf16 results after one more rounding).

Attention, per output: the result is rounded to bf16 (half a step: 2^-8 of its value), each
weight before the product with v to bf16 or, for the INT8 cache, fp16 (2^-8 or 2^-11 of itself, so of
mag = sum w|v| / sum w in all), and a score is off by e = (D + 8) 2^-23 max_j scale sum_d |q k|
(binary32 sums and products), which changes a weight by a factor within 1 +- 2e (numerator and
denominator). The exponential (2^-22), the sums and the joins of up to a few hundred parts stay
within 2^-15 of mag. fp16 weights are weight * value scale * 2^7 / M at the least, M a power of two
at most twice the largest value scale: below fp16's normal range they round to multiples of 2^-24, an
error of up to 2^-25 2^-7 M 127 <= 2^-31 max|v| per cache row beside the largest weight 1, which the
sum of the weights is at least. Bound: 1.02 (2^-8 |o| + mag (w + 4 e + 2^-15)) +
m 2^-31 max|v|, the factor for the cross term of the first two.
"""
import numpy as np
import pytest
import torch

from oracle import serve as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dq():
    import calibration_free_dual_b200 as pkg
    return pkg


@pytest.fixture(autouse=True)
def _clean(dq):
    yield
    assert dq.last_device_error() == 0


def _np(t):
    return t.detach().to(torch.float64).cpu().numpy()


def _x(rng, T, n, dtype, pad=0):
    x = rng.standard_normal((T, n + pad)).astype(np.float32)
    x[:, rng.choice(n, min(4, n), replace=False)] *= 50.0
    return torch.from_numpy(x).to(dtype).cuda()[:, :n]


# ------------------------------------------------------------------------- row quantizer
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,n,pad,with_c", [(1, 16, 0, False), (3, 80, 16, True),
                                            (700, 1280, 0, True), (5, 4096, 8, True),
                                            (333, 4112, 0, False), (2, 14336, 0, True),
                                            (600, 11008, 0, True), (3, 20000, 32, True),
                                            (500, 16400, 16, True), (7, 32768, 0, False), (3, 32784, 0, True)])
def test_row_quant_bit_exact(dq, dtype, T, n, pad, with_c):
    rng = np.random.default_rng(T + n)
    X = _x(rng, T, n, dtype, pad)
    if T > 2:
        X[1] = 0.0
        X[2] *= 2.0 ** -120
    c = torch.from_numpy(rng.uniform(0.25, 3.0, n).astype(np.float32)).cuda() if with_c else None
    r = dq.row_quant(X, c)
    q, d = O.row_quant(_np(X), None if c is None else _np(c))
    np.testing.assert_array_equal(r["codes"].cpu().numpy(), q)
    np.testing.assert_array_equal(_np(r["scales"]), d)


def test_row_quant_range_ends(dq):
    X = torch.zeros(6, 32, dtype=torch.float32)
    X[0, 3] = 1e-45                       # below the smallest scale's half: code 0, scale 2^-126
    X[1] = torch.finfo(torch.float32).max
    X[2] = -torch.finfo(torch.float32).max
    X[3, ::2] = -0.0
    X[4] = 2.0 ** -126
    X[5] = torch.arange(32) - 15.5
    r = dq.row_quant(X.cuda())
    q, d = O.row_quant(_np(X))
    np.testing.assert_array_equal(r["codes"].cpu().numpy(), q)
    np.testing.assert_array_equal(_np(r["scales"]), d)


@pytest.mark.parametrize("n", [64, 17408])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_row_quant_nonfinite(dq, n, bad):
    X = torch.ones(5, n, dtype=torch.bfloat16)
    X[3, n - 7] = bad
    r = dq.row_quant(X.cuda())
    assert dq.last_device_error() == 5
    s = _np(r["scales"])
    assert np.isnan(s[3]) and np.all(np.isfinite(np.delete(s, 3)))
    codes = r["codes"].cpu().numpy()
    assert np.all(codes[3] == 0) and np.all(np.delete(codes, 3, 0) == 127)


# --------------------------------------------------------------------------- INT8 product
def _operand(rng, rows, K, extreme=False):
    q = rng.integers(-127, 128, (rows, K)).astype(np.int8)
    if extreme:
        q[:] = 127
        q[::2] = -127
    s = rng.uniform(0.5, 1.5, rows).astype(np.float32) * np.float32(1e-3)
    return q, s, dict(codes=torch.from_numpy(q).cuda(), scales=torch.from_numpy(s).cuda())


GEMMS = [(1, 1, 16), (1, 8, 16), (1, 4096, 4096), (2, 130, 272), (7, 257, 144), (16, 1000, 2048),
         (33, 130, 272), (64, 128, 128), (65, 64, 400), (128, 128, 128), (129, 257, 4096),
         (200, 136, 336), (300, 520, 1040), (513, 1100, 640), (257, 300, 14336), (1025, 2050, 256)]


@pytest.mark.parametrize("T,N,K", GEMMS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gemm_bit_exact(dq, T, N, K, dtype):
    rng = np.random.default_rng(T + N + K)
    xq, xs, x = _operand(rng, T, K)
    wq, ws, w = _operand(rng, N, K)
    y = dq.w8a8_gemm(x, w, out_dtype=dtype)
    ref = torch.from_numpy(O.w8a8_gemm(xq, xs, wq, ws)).to(torch.float32).to(dtype)
    assert y.dtype == dtype and torch.equal(y.cpu(), ref)


@pytest.mark.parametrize("T,N", [(1, 24), (40, 130), (300, 300)])
def test_gemm_longest_sum(dq, T, N):
    """K = 131072 of +-127: the sum is just inside int32."""
    rng = np.random.default_rng(T)
    xq, xs, x = _operand(rng, T, 131072, extreme=True)
    wq, ws, w = _operand(rng, N, 131072, extreme=True)
    y = dq.w8a8_gemm(x, w)
    sign = np.where(np.arange(T)[:, None] % 2 == np.arange(N)[None, :] % 2, 1.0, -1.0)
    s = O.f32(xs.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :])
    np.testing.assert_array_equal(_np(y), O.f32(O.f32(sign * 127.0 * 127.0 * 131072) * s))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N,off,pitch", [(5, 66, 1, 75), (140, 130, 3, 201), (300, 256, 0, 260),
                                           (300, 256, 4, 264)])
def test_gemm_writes_only_its_rows(dq, dtype, T, N, off, pitch):
    """A result inside a wider buffer, from an odd element on: nothing else changes."""
    rng = np.random.default_rng(N)
    xq, xs, x = _operand(rng, T, 160)
    wq, ws, w = _operand(rng, N, 160)
    buf = torch.full((T + 2, pitch), 7.0, dtype=dtype, device="cuda")
    out = buf[1:T + 1, off:off + N]
    dq.w8a8_gemm(x, w, out_dtype=dtype, out=out)
    ref = torch.full((T + 2, pitch), 7.0, dtype=dtype)
    ref[1:T + 1, off:off + N] = torch.from_numpy(O.w8a8_gemm(xq, xs, wq, ws)).to(torch.float32).to(dtype)
    assert torch.equal(buf.cpu(), ref)


@pytest.mark.parametrize("T", [1, 4, 33, 200, 700])
@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.bfloat16),
                                             (torch.float32, torch.float32),
                                             (torch.bfloat16, torch.float32)])
def test_linear_is_row_quant_then_gemm(dq, T, dtype, out_dtype):
    rng = np.random.default_rng(T)
    K, N = 1296, 390
    X = _x(rng, T, K, dtype, 32)
    c = torch.from_numpy(rng.uniform(0.25, 3.0, K).astype(np.float32)).cuda()
    _, _, w = _operand(rng, N, K)
    y = dq.w8a8_linear(X, w, c, out_dtype=out_dtype)
    assert torch.equal(y, dq.w8a8_gemm(dq.row_quant(X, c), w, out_dtype=out_dtype))


def test_linear_approximates_the_layer(dq):
    """Weight and activation quantized with opposite column scales: W x within the two
    quantizers' steps (each at most half a step of its row: a / 254)."""
    rng = np.random.default_rng(3)
    T, N, K = 70, 200, 1024
    X, W = _x(rng, T, K, torch.bfloat16), _x(rng, N, K, torch.bfloat16)
    c = torch.from_numpy(rng.uniform(0.5, 2.0, K).astype(np.float32)).cuda()
    w = dq.row_quant(W, 1.0 / c)
    y = _np(dq.w8a8_linear(X, w, c, out_dtype=torch.float32))
    x, v = _np(X) * _np(c), _np(W) / _np(c)
    dx = np.abs(x).max(1) / 254.0 * 1.001
    dv = np.abs(v).max(1) / 254.0 * 1.001
    bound = (np.abs(x).sum(1)[:, None] * dv + dx[:, None] * np.abs(v).sum(1) + K * dx[:, None] * dv)
    assert np.all(np.abs(y - x @ v.T) <= bound * 1.001)


def test_linear_nonfinite_row_is_nan(dq):
    rng = np.random.default_rng(5)
    X = _x(rng, 6, 64, torch.bfloat16)
    X[4, 9] = float("nan")
    _, _, w = _operand(rng, 40, 64)
    y = dq.w8a8_linear(X, w)
    assert dq.last_device_error() == 5
    assert torch.isnan(y[4]).all() and torch.isfinite(y[[0, 1, 2, 3, 5]]).all()


# ----------------------------------------------------------------------------- append
def _tables(rng, rows, dim):
    a = rng.uniform(0, 6.28, (rows, dim // 2))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def _random_cache(rng, dq, pages, G, S, D, dtype, layout="head"):
    c = dq.kv_cache(pages, G, S, D, dtype=dtype)
    if layout == "token":                                # [pages, page_size, heads, D] underneath
        for n in ("k", "v"):
            c[n] = c[n].permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    elif layout == "pair":                               # k and v halves of one tensor
        both = torch.zeros((pages, 2, G, S, D), dtype=dtype, device="cuda")
        c["k"], c["v"] = both[:, 0], both[:, 1]
    for n in ("k", "v"):
        x = rng.standard_normal((pages, G, S, D))
        if dtype == torch.int8:
            c[n].copy_(torch.from_numpy(np.clip(np.rint(x * 40), -127, 127).astype(np.int8)))
            c[n + "_scales"].copy_(torch.from_numpy(
                (rng.uniform(0.2, 1.5, (pages, G, S)) / 40).astype(np.float32)))
        else:
            c[n].copy_(torch.from_numpy(x.astype(np.float32)))
    return c


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("T,H,G,D,S,dim,inter,layout",
                         [(1, 1, 1, 64, 16, 64, False, "head"), (5, 8, 2, 128, 16, 128, False, "token"),
                          (64, 32, 8, 128, 32, 64, False, "pair"), (77, 7, 1, 64, 64, 64, True, "head"),
                          (33, 12, 3, 128, 256, 24, True, "token"), (9, 4, 4, 64, 128, 0, False, "head"),
                          (200, 0, 5, 128, 16, 8, False, "head"), (700, 26, 6, 128, 32, 96, False, "token"),
                          (593, 7, 3, 64, 64, 32, True, "pair"), (20, 50, 2, 64, 16, 64, False, "head")])
def test_append_bit_exact(dq, dtype, kind, T, H, G, D, S, dim, inter, layout):
    rng = np.random.default_rng(T + H + G)
    pages = -(-T // S) + 3
    cache = _random_cache(rng, dq, pages, G, S, D, kind, layout)
    want = {n: _np(t).copy() for n, t in cache.items()}
    qkv = torch.from_numpy(rng.standard_normal((T, (H + 2 * G) * D + 8)).astype(np.float32)).to(dtype).cuda()
    qkv[0, :] = 0.0
    q = qkv[:, :H * D].view(T, H, D) if H else None
    k = qkv[:, H * D:(H + G) * D].view(T, G, D)
    v = qkv[:, (H + G) * D:(H + 2 * G) * D].view(T, G, D)
    slots = rng.permutation(pages * S)[:T].astype(np.int64)
    if T > 3:
        slots[2] = -1
        slots[T - 1] = -5
    rot, kr, qr = {}, _np(k), None if q is None else _np(q)
    if dim:
        cos, sin = _tables(rng, 50, dim)
        pos = rng.integers(0, 50, T).astype(np.int32)
        rot = dict(cos=torch.from_numpy(cos).cuda(), sin=torch.from_numpy(sin).cuda(),
                   positions=torch.from_numpy(pos).cuda(), interleaved=inter)
        kr = O.rotate(kr, cos, sin, pos, inter)
        qr = None if q is None else O.rotate(qr, cos, sin, pos, inter)
    got = dq.kv_append(k, v, cache, torch.from_numpy(slots).cuda(), q=q, **rot)
    for n, x in (("k", kr), ("v", _np(v))):
        if kind == torch.int8:
            codes, d = O.row_quant(x)
        else:
            codes = torch.from_numpy(x).to(torch.float32).to(torch.bfloat16).double().numpy()
        for t in range(T):
            if slots[t] >= 0:
                want[n][slots[t] // S, :, slots[t] % S] = codes[t]
                if kind == torch.int8:
                    want[n + "_scales"][slots[t] // S, :, slots[t] % S] = d[t]
    for n in cache:
        np.testing.assert_array_equal(_np(cache[n]), want[n], err_msg=n)
    if q is not None:
        assert torch.equal(got.cpu(), torch.from_numpy(qr).to(torch.float32).to(torch.bfloat16))


@pytest.mark.parametrize("T,H", [(11, 6), (11, 30), (650, 40)])
def test_append_rotates_queries_in_place(dq, T, H):
    rng = np.random.default_rng(1)
    G, D = 2, 64
    qkv = torch.from_numpy(rng.standard_normal((T, (H + 2 * G) * D)).astype(np.float32)).to(torch.bfloat16).cuda()
    q, k, v = (qkv[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, H), (H, H + G), (H + G, H + 2 * G)))
    cos, sin = _tables(rng, 30, D)
    rot = dict(cos=torch.from_numpy(cos).cuda(), sin=torch.from_numpy(sin).cuda(),
               positions=torch.arange(T, dtype=torch.int32, device="cuda") % 30)
    slots = torch.arange(T, device="cuda")
    pages = -(-T // 16)
    a = dq.kv_append(k, v, dq.kv_cache(pages, G, 16, D), slots, q=q, **rot)
    b = dq.kv_append(k, v, dq.kv_cache(pages, G, 16, D), slots, q=q, q_out=q, **rot)
    assert b.data_ptr() == q.data_ptr() and torch.equal(a, b)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("what", ["slot", "position_high", "position_low"])
def test_append_out_of_range_is_reported(dq, kind, what):
    """The token with the bad index writes nothing, the others are stored."""
    G, D, S, T = 2, 64, 16, 4
    cache = dq.kv_cache(2, G, S, D, dtype=kind)
    k = torch.ones(T, G, D, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([0, 1, 2, 3], device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    if what == "slot":
        slots[1] = 2 * S
    else:
        pos[1] = 5 if what == "position_high" else -1
    cos, sin = torch.ones(5, D // 2, device="cuda"), torch.zeros(5, D // 2, device="cuda")
    dq.kv_append(k, k, cache, slots, positions=pos, cos=cos, sin=sin)
    assert dq.last_device_error() == 1
    filled = _np(cache["k"]).reshape(2, G, S, D).any((1, 3))
    assert filled[0].tolist() == [True, False, True, True] + [False] * 12 and not filled[1].any()


def test_append_nonfinite_rows(dq):
    G, D = 2, 64
    k = torch.ones(3, G, D, dtype=torch.bfloat16, device="cuda")
    k[1, 1, 5] = float("inf")
    cache = dq.kv_cache(1, G, 16, D, dtype=torch.int8)
    dq.kv_append(k, torch.ones_like(k), cache, torch.arange(3, device="cuda"))
    assert dq.last_device_error() == 5
    s = _np(cache["k_scales"])[0]
    assert np.isnan(s[1, 1]) and np.isfinite(np.delete(s.ravel(), 16 + 1)).all()
    assert np.isfinite(_np(cache["v_scales"])).all()
    cache = dq.kv_cache(1, G, 16, D)
    dq.kv_append(k, k, cache, torch.arange(3, device="cuda"))       # bf16: stored as it is
    assert np.isinf(_np(cache["k"])[0, 1, 1, 5])


# -------------------------------------------------------------------------- attention
def _value(cache, n):
    x = _np(cache[n])
    return x * _np(cache[n + "_scales"])[..., None] if n + "_scales" in cache else x


def _setup(rng, dq, news, lens, H, G, D, S, kind, layout="head", spread=1.5):
    B = len(lens)
    used = [-(-m // S) for m in lens]
    pages = sum(used) + 3
    cache = _random_cache(rng, dq, pages, G, S, D, kind, layout)
    order = rng.permutation(pages)
    width = max(max(used), 1)
    # entries past a sequence's pages are never read
    table = np.full((B, width + 2), 2 ** 31 - 1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
    q = torch.from_numpy((rng.standard_normal((sum(news), H, D)) * spread).astype(np.float32)).to(torch.bfloat16).cuda()
    starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    return (q, cache, torch.from_numpy(table).cuda()[:, :width],
            torch.tensor(lens, dtype=torch.int32, device="cuda"),
            torch.from_numpy(starts).cuda(), table[:, :width])


def _poison(cache, table, lens, S):
    """NaN in every cache row that no sequence holds."""
    live = np.zeros(cache["k"].shape[0] * S, dtype=bool)
    for b, m in enumerate(lens):
        for j in range(m):
            live[table[b, j // S] * S + j % S] = True
    dead = torch.from_numpy(~live.reshape(-1, S)).cuda()
    for n in ("k", "v"):
        if n + "_scales" in cache:
            cache[n + "_scales"][dead[:, None, :].expand(-1, cache["k"].shape[1], -1)] = float("nan")
            cache[n][dead[:, None, :].expand(-1, cache["k"].shape[1], -1)] = -128
        else:
            cache[n][dead[:, None, :].expand(-1, cache["k"].shape[1], -1)] = float("nan")


def _check_attention(o, q, cache, table, lens, news, causal, scale=None):
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    kv = [np.nan_to_num(_value(cache, n)) for n in ("k", "v")]
    S = cache["k"].shape[2]
    w = 2.0 ** -8 if cache["k"].dtype == torch.bfloat16 else 2.0 ** -11
    at = 0
    got, qn = _np(o), _np(q)
    for b, (n, m) in enumerate(zip(news, lens)):
        k, v = (x[table[b, :-(-m // S)]].transpose(0, 2, 1, 3).reshape(-1, x.shape[1], D)[:m] for x in kv)
        ref, mag, dot = O.attention(qn[at:at + n], k, v, causal, scale)
        e = (D + 8) * 2.0 ** -23 * dot[..., None]
        # every weight over their sum moves by a factor within exp(+-2e), and exp(2e) - 1 <= 4e up to
        # e = 0.6 (exp(1.2) - 1 = 2.32 < 2.4; convex, equal at 0)
        assert e.max(initial=0.0) < 0.6
        bound = 1.02 * (2.0 ** -8 * np.abs(ref) + mag * (w + 4 * e + 2.0 ** -15)) + m * 2.0 ** -31 * np.abs(v).max(initial=0.0)
        err = np.abs(got[at:at + n] - ref)
        assert np.all(err <= bound), (b, n, m, float(np.nanmax(err / np.maximum(bound, 1e-30))))
        at += n


# (new tokens, lengths): single tokens, short and long; lengths around tiles and pages
DECODES = [([1], [1]), ([1] * 5, [17, 0, 1, 16, 300]), ([1] * 3, [4097, 64, 2000])]
CHUNKS = [([3], [3]), ([2, 1, 5, 0, 9], [40, 1, 4, 0, 33]), ([16, 31], [512, 31]),
          ([17, 130], [700, 131]), ([200], [1111]), ([64, 1, 128, 65], [64, 1000, 129, 400]),
          ([300, 5], [300, 2500])]
HEADS = [(1, 1, 64), (8, 2, 64), (32, 8, 128), (7, 1, 128), (4, 4, 128), (16, 1, 64)]


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("H,G,D", HEADS)
@pytest.mark.parametrize("news,lens", DECODES + CHUNKS)
def test_attention(dq, kind, H, G, D, news, lens):
    rng = np.random.default_rng(sum(lens) + H + D)
    S = [16, 32, 64, 128, 256][(sum(lens) + H) % 5]
    q, cache, table, lt, st, tn = _setup(rng, dq, news, lens, H, G, D, S, kind)
    _poison(cache, tn, lens, S)
    o = dq.paged_attention(q, cache, table, lt, q_starts=st, max_q=max(news), max_len=max(lens))
    _check_attention(o, q, cache, tn, lens, news, True)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("S", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["head", "token", "pair"])
@pytest.mark.parametrize("n", [1, 90, 300])
def test_attention_page_sizes_and_layouts(dq, kind, S, layout, n):
    rng = np.random.default_rng(S + n)
    news, lens = [n, n], [n + 301, n]
    q, cache, table, lt, st, tn = _setup(rng, dq, news, lens, 4, 2, 128, S, kind, layout)
    _poison(cache, tn, lens, S)
    o = dq.paged_attention(q, cache, table, lt, q_starts=st, max_q=n)
    _check_attention(o, q, cache, tn, lens, news, True)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("news,lens", [([4, 2], [9, 300]), ([12, 5], [9, 1300]), ([150, 3], [77, 500])])
def test_attention_not_causal(dq, kind, news, lens):
    rng = np.random.default_rng(9)
    q, cache, table, lt, st, tn = _setup(rng, dq, news, lens, 8, 2, 64, 16, kind)
    _poison(cache, tn, lens, 16)
    o = dq.paged_attention(q, cache, table, lt, q_starts=st, causal=False, scale=0.2)
    _check_attention(o, q, cache, tn, lens, news, False, 0.2)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("n", [1, 5, 22, 150])
def test_attention_rows_without_keys_are_zero(dq, kind, n):
    """More new tokens than cache rows: the first see nothing; an empty sequence gives zeros."""
    rng = np.random.default_rng(n)
    news, lens = [n, n], [n // 2, 0]
    q, cache, table, lt, st, tn = _setup(rng, dq, news, lens, 4, 2, 64, 16, kind)
    _poison(cache, tn, lens, 16)
    o = dq.paged_attention(q, cache, table, lt, q_starts=st, max_len=3000 if n == 1 else None
                           ) if n != 1 else dq.paged_attention(q, cache, table, lt)
    _check_attention(o, q, cache, tn, lens, news, True)
    assert (o[n:] == 0).all() and (o[:n - n // 2] == 0).all()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("n", [1, 40])
def test_attention_value_scales_of_all_sizes(dq, kind, n):
    """Value rows whose sizes span 2^-60 .. 2^40, scores that span hundreds: fp16 weights keep up."""
    rng = np.random.default_rng(n)
    news, lens = [n], [700]
    q, cache, table, lt, st, tn = _setup(rng, dq, news, lens, 4, 2, 128, 32, kind, spread=6.0)
    f = np.exp2(np.where(np.arange(32) % 2, rng.integers(-60, 0, 32), rng.integers(0, 41, 32))).astype(np.float32)
    f = torch.from_numpy(np.minimum(f, 2.0 ** 30)).cuda()
    if kind == torch.int8:
        cache["v_scales"] *= f
    else:
        cache["v"] *= f[:, None].to(torch.bfloat16)
    o = dq.paged_attention(q, cache, table, lt, q_starts=st)
    _check_attention(o, q, cache, tn, lens, news, True)


def test_attention_queries_of_all_sizes(dq):
    """INT8 cache: query rows from 2^-100 to 2^100 (keys scaled the other way), zero rows."""
    rng = np.random.default_rng(2)
    news, lens = [6], [300]
    q, cache, table, lt, st, tn = _setup(rng, dq, news, lens, 2, 1, 64, 16, torch.int8)
    for e in (-100, 100):
        q2 = q * 2.0 ** e
        q2[3] = 0.0
        c2 = dict(cache, k_scales=cache["k_scales"] * 2.0 ** -e)
        o = dq.paged_attention(q2, c2, table, lt, q_starts=st)
        _check_attention(o, q2, c2, tn, lens, news, True)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("n", [1, 70])
def test_attention_writes_only_its_rows(dq, kind, n):
    """Rows behind the last sequence and between the heads of a wider buffer stay."""
    rng = np.random.default_rng(4)
    news, lens = [n, n], [200, 333]
    q, cache, table, lt, st, tn = _setup(rng, dq, news, lens, 4, 2, 64, 16, kind)
    q = torch.cat([q, torch.full_like(q[:3], float("nan"))])
    buf = torch.full((q.shape[0], 4 * 64 + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, 8:8 + 256].view(-1, 4, 64)
    dq.paged_attention(q, cache, table, lt, q_starts=st, max_q=n, out=out)
    _check_attention(out[:2 * n], q[:2 * n], cache, tn, lens, news, True)
    assert (buf[:, :8] == 7).all() and (buf[:, 264:] == 7).all() and (buf[2 * n:] == 7).all()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("n", [1, 33])
def test_attention_bad_pages_and_bounds_are_reported(dq, kind, n):
    rng = np.random.default_rng(6)
    news, lens = [n, n], [200, 120]
    q, cache, table, lt, st, tn = _setup(rng, dq, news, lens, 4, 2, 64, 16, kind)
    good = dq.paged_attention(q, cache, table, lt, q_starts=st, max_q=n)
    assert dq.last_device_error() == 0
    for bad in (-1, cache["k"].shape[0], 2 ** 31 - 1, -2 ** 31):
        t2 = table.clone()
        t2[1, 3] = bad
        o = dq.paged_attention(q, cache, t2, lt, q_starts=st, max_q=n)
        assert dq.last_device_error() == 1
        assert torch.equal(o[:n], good[:n])                    # the other sequence is untouched
    for l2 in (-1, 16 * table.shape[1] + 1):
        lens2 = lt.clone()
        lens2[0] = l2
        t2 = torch.zeros_like(table)
        dq.paged_attention(q, cache, t2, lens2, q_starts=st, max_q=n)
        assert dq.last_device_error() == 1
    for s2 in ([0, n, 2 * n + 1], [0, -4, 2 * n], [n, 0, 2 * n]):
        dq.paged_attention(q, cache, table, lt, q_starts=torch.tensor(s2, dtype=torch.int32, device="cuda"), max_q=n)
        assert dq.last_device_error() == 1


def test_attention_many_sequences_share_pages(dq):
    """A prefix shared by two sequences: the same pages in both tables."""
    rng = np.random.default_rng(8)
    news, lens = [1, 1], [96, 80]
    q, cache, table, lt, st, tn = _setup(rng, dq, news, lens, 4, 2, 64, 16, torch.int8)
    table[1, :4] = table[0, :4]
    tn = table.cpu().numpy()
    o = dq.paged_attention(q, cache, table, lt)
    _check_attention(o, q, cache, tn, lens, news, True)


# ------------------------------------------------------------ the operators as they are used
class _Block:
    """One attention block: quantized projection, append, attention, quantized projection."""

    def __init__(self, dq, rng, hidden, H, G, D, kind, pages, S):
        self.dq, self.H, self.G, self.D = dq, H, G, D
        self.c = [torch.from_numpy(rng.uniform(0.5, 2.0, n).astype(np.float32)).cuda() for n in (hidden, H * D)]
        W = [torch.from_numpy((rng.standard_normal(s) / np.sqrt(s[1])).astype(np.float32)).cuda()
             for s in (((H + 2 * G) * D, hidden), (hidden, H * D))]
        self.w = [dq.row_quant(w, 1.0 / c) for w, c in zip(W, self.c)]
        cos, sin = _tables(rng, 4096, D)
        self.rot = dict(cos=torch.from_numpy(cos).cuda(), sin=torch.from_numpy(sin).cuda())
        self.cache = dq.kv_cache(pages, G, S, D, dtype=kind)

    def __call__(self, x, slots, positions, table, lengths, starts, max_q, max_len):
        dq, H, G, D, T = self.dq, self.H, self.G, self.D, x.shape[0]
        qkv = dq.w8a8_linear(x, self.w[0], self.c[0])
        q, k, v = (qkv[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, H), (H, H + G), (H + G, H + 2 * G)))
        q = dq.kv_append(k, v, self.cache, slots, positions=positions, q=q, q_out=q, **self.rot)
        o = dq.paged_attention(q, self.cache, table, lengths, q_starts=starts, max_q=max_q, max_len=max_len)
        return qkv, q, o, dq.w8a8_linear(o.view(T, H * D), self.w[1], self.c[1])


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.int8])
def test_attention_block_prompt_then_tokens(dq, kind):
    """Two sequences through prompt, chunk and single tokens; each step against the oracle from
    the step's own inputs, then the same single-token steps replayed from a captured graph."""
    rng = np.random.default_rng(12)
    hidden, H, G, D, S, pages = 256, 8, 2, 64, 16, 40
    blk = _Block(dq, rng, hidden, H, G, D, kind, pages, S)
    table = torch.from_numpy(rng.permutation(pages).reshape(2, 20).astype(np.int32)).cuda()
    tn = table.cpu().numpy()
    done = [0, 0]

    def inputs(news):
        pos = np.concatenate([np.arange(d, d + n) for d, n in zip(done, news)]).astype(np.int32)
        slots = np.concatenate([tn[b, np.arange(d, d + n) // S].astype(np.int64) * S + np.arange(d, d + n) % S
                                for b, (d, n) in enumerate(zip(done, news))])
        for b in range(2):
            done[b] += news[b]
        x = _x(rng, sum(news), hidden, torch.bfloat16)
        starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        return [x] + [torch.from_numpy(a).cuda() for a in (slots, pos)] + [
            table, torch.tensor(done, dtype=torch.int32, device="cuda"), torch.from_numpy(starts).cuda()]

    def check(args, res, news):
        qkv, q, o, y = res
        x = _np(args[0])
        xq, xs = O.row_quant(x, _np(blk.c[0]))
        ref = O.w8a8_gemm(xq, xs, _np(blk.w[0]["codes"]).astype(np.int64), _np(blk.w[0]["scales"]))
        ref = torch.from_numpy(ref).float().bfloat16()
        assert torch.equal(qkv[:, H * D:].cpu(), ref[:, H * D:])          # (q has been rotated in place)
        cs, sn = (_np(blk.rot[n]) for n in ("cos", "sin"))
        pos = args[2].cpu().numpy()
        qr = O.rotate(ref[:, :H * D].double().numpy().reshape(-1, H, D), cs, sn, pos)
        assert torch.equal(q.cpu(), torch.from_numpy(qr).float().bfloat16())
        _check_attention(o, q, blk.cache, tn, done, news, True)
        oq, os_ = O.row_quant(_np(o).reshape(-1, H * D), _np(blk.c[1]))
        yr = O.w8a8_gemm(oq, os_, _np(blk.w[1]["codes"]).astype(np.int64), _np(blk.w[1]["scales"]))
        assert torch.equal(y.cpu(), torch.from_numpy(yr).float().bfloat16())

    for news in ([37, 150], [70, 3], [1, 1]):
        a = inputs(news)
        check(a, blk(*a, max(news), 320), news)
    # a captured step, replayed over new contents of the same tensors
    a = inputs([1, 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        blk(*a, 1, 320)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = blk(*a, 1, 320)
    graph.replay()
    check(a, res, [1, 1])
    for _ in range(3):
        for t, n in zip(a, inputs([1, 1])):
            t.copy_(n)
        graph.replay()
        check(a, res, [1, 1])


@pytest.mark.parametrize("T", [1, 200])
def test_calls_on_another_stream(dq, T):
    """Every helper on a stream of its own gives what it gives on the current one, also while the
    current stream is busy with the same operators."""
    rng = np.random.default_rng(T)
    X = _x(rng, T, 512, torch.bfloat16)
    _, _, w = _operand(rng, 256, 512)
    news, lens = [T], [T + 500]
    q, cache, table, lt, st, tn = _setup(rng, dq, news, lens, 4, 2, 64, 16, torch.int8)
    kv = _x(rng, T, 128, torch.bfloat16).view(T, 2, 64)
    slots = torch.arange(T, device="cuda")
    c2 = [dq.kv_cache(20, 2, 16, 64, dtype=torch.int8) for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    res = []
    for i, stream in enumerate((s, None)):
        kw = dict(stream=stream)
        got = [dq.w8a8_linear(X, w, **kw), dq.w8a8_gemm(dq.row_quant(X, **kw), w, **kw),
               dq.paged_attention(q, cache, table, lt, q_starts=st, **kw)]
        dq.kv_append(kv, kv, c2[i], slots, **kw)
        res.append(got + [c2[i]["k"], c2[i]["v_scales"]])
    torch.cuda.synchronize()
    for x, y in zip(*res):
        assert torch.equal(x, y)


def test_two_calls_share_one_workspace_in_stream_order(dq):
    rng = np.random.default_rng(1)
    news, lens = [1, 1], [3000, 2000]
    q, cache, table, lt, st, tn = _setup(rng, dq, news, lens, 4, 2, 64, 16, torch.bfloat16)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    a = dq.paged_attention(q, cache, table, lt, workspace=ws)
    b = dq.paged_attention(q.flip(0).contiguous(), cache, table.flip(0).contiguous(), lt.flip(0).contiguous(), workspace=ws)
    assert torch.equal(a, b.flip(0))


# ------------------------------------------------------------------- calls around the edges
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("n", [1, 60, 300])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-6])
def test_attention_odd_scales(dq, kind, n, scale):
    rng = np.random.default_rng(n)
    news, lens = [n], [n + 100]
    q, cache, table, lt, st, tn = _setup(rng, dq, news, lens, 4, 2, 128, 32, kind)
    _poison(cache, tn, lens, 32)
    o = dq.paged_attention(q, cache, table, lt, q_starts=st, scale=scale)
    _check_attention(o, q, cache, tn, lens, news, True, scale)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("n", [1, 70])
def test_split_attention_in_a_graph(dq, kind, n):
    """Sequences split over CTAs and joined, captured and replayed over new queries, new lengths and
    a new table in the same tensors."""
    rng = np.random.default_rng(n)
    news, lens = [n, n], [6000, 4001]
    q, cache, table, lt, st, tn = _setup(rng, dq, news, lens, 8, 2, 128, 64, kind)
    kw = dict(q_starts=st, max_q=n, max_len=6000)
    dq.paged_attention(q, cache, table, lt, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = dq.paged_attention(q, cache, table, lt, **kw)
    for lens in ([6000, 4001], [n, 5999]):
        table.copy_(torch.from_numpy(tn).cuda() % cache["k"].shape[0])
        lt.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(torch.from_numpy(rng.standard_normal(q.shape).astype(np.float32)).to(torch.bfloat16))
        graph.replay()
        _check_attention(o, q, cache, table.cpu().numpy(), lens, news, True)


def test_products_and_attention_on_two_streams(dq):
    """Kernels that share SMs, tensor memory and clusters, at once on two streams: the same results
    as one after the other, and both end."""
    rng = np.random.default_rng(0)
    _, _, w = _operand(rng, 4096, 512)
    _, _, small = _operand(rng, 1024, 256)
    X, x = _x(rng, 2048, 512, torch.bfloat16), _x(rng, 5, 256, torch.bfloat16)
    news, lens = [300, 1], [900, 3000]
    q, cache, table, lt, st, tn = _setup(rng, dq, news, lens, 8, 2, 128, 32, torch.int8)
    calls = [lambda s: dq.w8a8_linear(X, w, stream=s), lambda s: dq.w8a8_linear(x, small, stream=s),
             lambda s: dq.paged_attention(q, cache, table, lt, q_starts=st, max_q=300, stream=s),
             lambda s: dq.paged_attention(q[300:], cache, table[1:], lt[1:], stream=s)]
    want = [f(None) for f in calls]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for i in range(24):
        for s, f in ((a, i % 4), (b, (i + 1 + i // 4) % 4)):
            got.append((f, calls[f](s)))
    torch.cuda.synchronize()
    for f, y in got:
        assert torch.equal(y, want[f])


def test_empty_calls(dq):
    X = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    r = dq.row_quant(X)
    assert r["codes"].shape == (0, 64) and r["scales"].shape == (0,)
    w = dict(codes=torch.ones(8, 64, dtype=torch.int8, device="cuda"), scales=torch.ones(8, device="cuda"))
    assert dq.w8a8_gemm(r, w).shape == (0, 8) and dq.w8a8_linear(X, w).shape == (0, 8)
    cache = dq.kv_cache(2, 2, 16, 64)
    kv = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    e64 = torch.empty(0, dtype=torch.int64, device="cuda")
    assert dq.kv_append(kv, kv, cache, e64) is None
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    assert dq.paged_attention(q, cache, torch.empty(0, 3, **i32), torch.empty(0, **i32)).shape == (0, 4, 64)
    # two sequences without a token, one without a cache row
    o = dq.paged_attention(torch.ones(1, 4, 64, dtype=torch.bfloat16, device="cuda"), cache, torch.zeros(3, 0, **i32),
                           torch.zeros(3, **i32), q_starts=torch.tensor([0, 0, 1, 1], **i32))
    assert (o == 0).all()


def test_helpers_refuse_bad_tensors(dq):
    dev = dict(device="cuda")
    X = torch.ones(4, 64, dtype=torch.bfloat16, **dev)
    w = dict(codes=torch.ones(8, 64, dtype=torch.int8, **dev), scales=torch.ones(8, **dev))
    for bad in (X.t(), X[0], X.expand(2, 4, 64)):
        with pytest.raises(ValueError):
            dq.row_quant(bad)
    with pytest.raises(dq.DQError):
        dq.row_quant(X[:1].expand(4, 64))                       # rows on top of one another
    with pytest.raises(dq.DQError):
        dq.row_quant(X[:, 1:49])                                # 2-byte aligned
    with pytest.raises(TypeError):
        dq.row_quant(X.half())
    with pytest.raises(ValueError):
        dq.row_quant(X, torch.ones(63, **dev))
    with pytest.raises(TypeError):
        dq.row_quant(X, torch.ones(64, dtype=torch.bfloat16, **dev))
    with pytest.raises(TypeError):
        dq.w8a8_linear(X, w, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        dq.w8a8_linear(X[:, :48], w)
    with pytest.raises(TypeError):
        dq.w8a8_linear(X, dict(w, codes=w["codes"].to(torch.uint8)))
    with pytest.raises(ValueError):
        dq.w8a8_linear(X, dict(w, scales=w["scales"][:7]))
    with pytest.raises(ValueError):
        dq.w8a8_linear(X, w, out=torch.empty(4, 9, dtype=torch.bfloat16, **dev))
    with pytest.raises(ValueError):
        dq.w8a8_linear(X, w, workspace=torch.empty(8, dtype=torch.uint8, **dev))
    cache = dq.kv_cache(4, 2, 16, 64)
    kv = torch.ones(3, 2, 64, dtype=torch.bfloat16, **dev)
    slots = torch.arange(3, **dev)
    with pytest.raises(TypeError):
        dq.kv_append(kv, kv.float(), cache, slots)
    with pytest.raises(TypeError):
        dq.kv_append(kv, kv, cache, slots.int())
    with pytest.raises(ValueError):
        dq.kv_append(kv, kv[:2], cache, slots)
    with pytest.raises(ValueError):
        dq.kv_append(kv, kv, cache, slots, positions=slots.int())
    with pytest.raises(ValueError):
        dq.kv_append(kv, kv, cache, slots, q_out=kv)
    with pytest.raises(ValueError):
        dq.kv_append(kv, kv, dict(cache, v=cache["v"].transpose(1, 2).contiguous().transpose(1, 2)), slots)
    with pytest.raises(TypeError):
        dq.kv_append(kv, kv, dict(cache, v=cache["v"].float()), slots)
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, **dev)
    table, lens = torch.zeros(3, 4, dtype=torch.int32, **dev), torch.ones(3, dtype=torch.int32, **dev)
    with pytest.raises(TypeError):
        dq.paged_attention(q.float(), cache, table, lens)
    with pytest.raises(TypeError):
        dq.paged_attention(q, cache, table.long(), lens)
    with pytest.raises(ValueError):
        dq.paged_attention(q, cache, table[:2], lens[:2])
    with pytest.raises(ValueError):
        dq.paged_attention(q, cache, table, lens, max_len=65)
    with pytest.raises(ValueError):
        dq.paged_attention(q.transpose(0, 1).contiguous().transpose(0, 1), cache, table, lens)
    with pytest.raises(dq.DQError):
        dq.paged_attention(q[:, :3].contiguous(), cache, table, lens)   # 3 heads on 2 key heads
