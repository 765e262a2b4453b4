"""Timed cases of the 8-bit serving operators: the per-token quantizer, the 8-bit integer
products, the paged key/value cache and the attention that reads it.

`run` computes each operator in plain torch operations (binary32, rounded once at the end), or, where
`own` is set, calls the library. `exact` restates the definitions in 64 bits.

Definitions (fl32: one IEEE binary32 operation):
  rows    x~ = fl32(X * c); a = max |x~| of the row; d = max(fl32(a / 127), 2^-126), 0 for a = 0;
          q = RNE(fl32(x~ * fl32(1 / d))) within -127..127
  gemm    y[t, i] = xs[t] ws[i] sum_j qx[t, j] qw[i, j]
  linear  rows of X, then gemm with the weight's codes
  append  keys and queries rotated by their position, keys and values into the slots of a
          paged cache (bf16, or 8-bit codes with one scale per token and head, as `rows`)
  attend  softmax(scale q k) v of a batch of chunks of new tokens over their pages, causal
"""
import math

import numpy as np
import torch

own = False

Q_MAX = 127.0
TINY = 2.0 ** -126


# --------------------------------------------------------------------------------- cases
def listed():
    return [
        # the tokens of a small decode batch, quantized before a projection of the 8B shape
        {"name": "rows_decode", "op": "rows", "T": 16, "K": 4096, "x": "bf16", "c": True},
        # the activation workload of the benchmark: 8192 tokens x 4096 channels
        {"name": "rows_prompt", "op": "rows", "T": 8192, "K": 4096, "x": "bf16", "c": True},
        # up projection of the 7B shape on a ragged prompt, codes at hand, binary32 result
        {"name": "gemm_ragged", "op": "gemm", "T": 777, "N": 11008, "K": 4096, "y": "f32"},
        # gate projection of the 8B shape on a long prompt
        {"name": "gemm_prompt", "op": "gemm", "T": 8192, "N": 14336, "K": 4096, "y": "bf16"},
        # one token through the down projection of the 8B shape
        {"name": "linear_token", "op": "linear", "T": 1, "N": 4096, "K": 14336, "x": "bf16",
         "y": "bf16", "c": True},
        # a decode batch of odd size through the up projection of the 1B shape, binary32
        {"name": "linear_batch", "op": "linear", "T": 45, "N": 8192, "K": 2048, "x": "f32",
         "y": "f32", "c": False},
        # one new token of each of 64 sequences into an 8-bit cache
        {"name": "append_decode", "op": "append", "T": 64, "H": 32, "G": 8, "D": 128,
         "page": 16, "cache": "int8", "skip": 0.05},
        # a prompt batch into a bf16 cache, as many key heads as query heads
        {"name": "append_prompt", "op": "append", "T": 6001, "H": 32, "G": 32, "D": 128,
         "page": 64, "cache": "bf16", "skip": 0.0},
        # one user: single token over a short context, heads of the 1B shape
        {"name": "attend_token", "op": "attend", "B": 1, "new": 1, "even": True, "ctx": 611,
         "H": 32, "G": 8, "D": 64, "page": 16, "cache": "bf16"},
        # a decode batch over long ragged contexts in an 8-bit cache, heads of the 8B shape
        {"name": "attend_decode", "op": "attend", "B": 48, "new": 1, "even": True,
         "ctx": 16000, "H": 32, "G": 8, "D": 128, "page": 32, "cache": "int8"},
        # a long prompt taken in chunks: 1000 new tokens over 24000 keys
        {"name": "attend_chunk", "op": "attend", "B": 1, "new": 1000, "even": True,
         "ctx": 24000, "H": 32, "G": 8, "D": 128, "page": 64, "cache": "bf16"},
        # a mixed batch: chunks from one token to 2500, heads of the 7B shape, 8-bit cache
        {"name": "attend_mixed", "op": "attend", "B": 5, "new": 2500, "even": False,
         "ctx": 4100, "H": 32, "G": 32, "D": 128, "page": 128, "cache": "int8"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows", "gemm", "linear", "append", "attend", "attend"])
    if op == "rows":
        return {"op": op, "T": _log(rng, 1, 8000), "K": 16 * _log(rng, 4, 256),
                "x": rng.choice(["bf16", "f32"]), "c": rng.random() < 0.5}
    if op in ("gemm", "linear"):
        case = {"op": op, "T": _log(rng, 1, 6000), "N": _log(rng, 64, 9000),
                "K": 16 * _log(rng, 8, 512), "y": rng.choice(["bf16", "f32"])}
        if op == "linear":
            case.update(x=rng.choice(["bf16", "f32"]), c=rng.random() < 0.5)
        return case
    G = rng.choice([1, 2, 4, 8])
    case = {"op": op, "H": G * rng.choice([1, 2, 4, 7, 8]), "G": G, "D": rng.choice([64, 128]),
            "page": rng.choice([16, 32, 64, 128, 256]), "cache": rng.choice(["bf16", "int8"])}
    if op == "append":
        case.update(T=_log(rng, 1, 6000), skip=rng.choice([0.0, 0.1]))
        return case
    new, B = rng.choice([(1, _log(rng, 1, 40)), (_log(rng, 2, 16), _log(rng, 1, 24)),
                         (_log(rng, 17, 400), _log(rng, 1, 3))])
    case.update(B=B, new=new, even=rng.random() < 0.5, ctx=new + _log(rng, 1, 14000))
    return case


def work(case):
    op = case["op"]
    if op == "rows":
        T, K = case["T"], case["K"]
        return {"bytes": T * K * (_size(case["x"]) + 1) + 4 * T + 4 * K * case["c"],
                "flops": 3 * T * K}
    if op in ("gemm", "linear"):
        T, N, K = case["T"], case["N"], case["K"]
        xb = 1 if op == "gemm" else _size(case["x"])
        return {"bytes": T * K * xb + N * K + T * N * _size(case["y"]) + 4 * (T + N),
                "flops": 2 * T * N * K}
    row = 2 * case["D"] if case["cache"] == "bf16" else case["D"] + 4
    if op == "append":
        T, H, G, D = case["T"], case["H"], case["G"], case["D"]
        return {"bytes": T * (4 * H * D + 4 * G * D + 2 * G * row + 4 * D + 12),
                "flops": 3 * T * (H + G) * D}
    news, lens = _lengths(case)
    H, G, D = case["H"], case["G"], case["D"]
    pairs = sum(n * s - n * (n - 1) // 2 for n, s in zip(news, lens))
    return {"bytes": sum(lens) * G * 2 * row + sum(news) * H * D * 4,
            "flops": 4 * H * D * pairs}


# -------------------------------------------------------------------------------- inputs
def _size(t):
    return 2 if t == "bf16" else 4


def _type(t):
    return torch.bfloat16 if t == "bf16" else torch.float32


def _lengths(case):
    """New tokens and keys in all of each sequence: the case's, or spread from one up to it."""
    B, new, ctx = case["B"], case["new"], case["ctx"]
    if case["even"]:
        news = [new] * B
    else:
        news = [1 + (new - 1) * i // max(1, B - 1) for i in range(B)]
    if B == 1:
        return news, [ctx]
    # contexts from a quarter of the longest up to it, in no order
    lens = [ctx - (ctx * 3 // 4) * ((i * 7) % B) // B for i in range(B)]
    return news, [max(n, s) for n, s in zip(news, lens)]


def _activations(g, T, K, dtype):
    # unit normal channels, six of them fifty times as large
    x = torch.randn((T, K), generator=g, device="cuda")
    x[:, torch.randperm(K, generator=g, device="cuda")[:6]] *= 50.0
    return x.to(dtype)


def _codes(g, rows, K):
    q = (torch.randn((rows, K), generator=g, device="cuda") * 32.0).round().clamp(-127, 127)
    s = (torch.rand((rows,), generator=g, device="cuda") + 0.5) * 5e-4
    return {"codes": q.to(torch.int8), "scales": s}


def _cache(g, pages, G, page, D, kind):
    c = {}
    for name, spread in (("k", 1.0), ("v", 1.0)):
        x = torch.randn((pages, G, page, D), generator=g, device="cuda") * spread
        if kind == "bf16":
            c[name] = x.to(torch.bfloat16)
        else:
            c[name] = (x * 36.0).round().clamp(-127, 127).to(torch.int8)
            c[name + "_scales"] = (torch.rand((pages, G, page), generator=g, device="cuda")
                                   + 0.5) / 36.0
    return c


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"case": dict(case)}
    if op == "rows":
        s["X"] = _activations(g, case["T"], case["K"], _type(case["x"]))
    elif op == "gemm":
        s["x"] = _codes(g, case["T"], case["K"])
        s["w"] = _codes(g, case["N"], case["K"])
    elif op == "linear":
        s["X"] = _activations(g, case["T"], case["K"], _type(case["x"]))
        s["w"] = _codes(g, case["N"], case["K"])
    if op in ("rows", "linear"):
        # column scales around one, as the solver returns them
        s["c"] = (torch.randn((case["K"],), generator=g, device="cuda") * 0.3).exp() \
            if case["c"] else None
    if op == "append":
        T, H, G, D, page = case["T"], case["H"], case["G"], case["D"], case["page"]
        # q, k and v are the columns of one projection's result
        qkv = torch.randn((T, (H + 2 * G) * D), generator=g, device="cuda").to(torch.bfloat16)
        s["q"] = qkv[:, :H * D].view(T, H, D)
        s["k"] = qkv[:, H * D:(H + G) * D].view(T, G, D)
        s["v"] = qkv[:, (H + G) * D:].view(T, G, D)
        pages = -(-T // page) + 7
        s["cache"] = _cache(g, pages, G, page, D, case["cache"])
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
        drop = torch.rand((T,), generator=g, device="cuda") < case["skip"]
        s["slots"] = torch.where(drop, -torch.ones_like(slots), slots)   # padding tokens
        limit = 8192
        s["positions"] = torch.randint(0, limit, (T,), generator=g, device="cuda",
                                       dtype=torch.int32)
        freq = 500000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
        angle = torch.arange(limit, device="cuda", dtype=torch.float64)[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    if op == "attend":
        news, lens = _lengths(case)
        H, G, D, page = case["H"], case["G"], case["D"], case["page"]
        width = -(-max(lens) // page)
        used = sum(-(-n // page) for n in lens)
        s["cache"] = _cache(g, used + 5, G, page, D, case["cache"])
        order = torch.randperm(used + 5, generator=g, device="cuda").to(torch.int32)
        table, at = torch.zeros((case["B"], width), dtype=torch.int32, device="cuda"), 0
        for b, n in enumerate(lens):
            k = -(-n // page)
            table[b, :k] = order[at:at + k]
            at += k
        s["table"] = table
        s["starts"] = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32,
                                   device="cuda")
        s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["max_new"], s["max_len"] = max(news), max(lens)
        q = torch.randn((sum(news), H, D), generator=g, device="cuda")
        s["q"] = (q * 2.0).to(torch.bfloat16)
    return s


# --------------------------------------------------------------------------- plain forms
def _plain_rows(x):
    """Codes (as binary32 integers) and scale of each row (last axis) of a binary32 tensor."""
    a = x.abs().amax(-1, keepdim=True)
    d = torch.maximum(a / torch.full_like(a, Q_MAX), torch.full_like(a, TINY))
    q = (x * torch.reciprocal(d)).round().clamp(-Q_MAX, Q_MAX)
    zero = a == 0
    return torch.where(zero, torch.zeros_like(q), q), torch.where(zero, a, d).squeeze(-1)


def _plain_product(qx, xs, w, dtype):
    y = qx @ w["codes"].float().t()
    return (y * (xs[:, None] * w["scales"][None, :])).to(dtype)


def _plain_rotate(x, cos, sin):
    x = x.float()
    a, b = x.chunk(2, -1)
    cos, sin = cos[:, None, :], sin[:, None, :]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(s):
    cache, slots = s["cache"], s["slots"]
    pos = s["positions"].long()
    cos, sin = s["cos"][pos], s["sin"][pos]
    keep = slots >= 0
    page = s["case"]["page"]
    at, row = slots[keep] // page, slots[keep] % page
    for name, x in (("k", _plain_rotate(s["k"], cos, sin)), ("v", s["v"].float())):
        if s["case"]["cache"] == "bf16":
            cache[name][at, :, row] = x[keep].to(torch.bfloat16)
        else:
            q, d = _plain_rows(x[keep])
            cache[name][at, :, row] = q.to(torch.int8)
            cache[name + "_scales"][at, :, row] = d
    return {"q": _plain_rotate(s["q"], cos, sin).to(torch.bfloat16), **cache}


def _plain_gather(s, name):
    """[B, keys, G, D] in binary32: every sequence's pages in order."""
    cache, table = s["cache"], s["table"].long()
    x = cache[name][table].float()                       # [B, width, G, page, D]
    if name + "_scales" in cache:
        x = x * cache[name + "_scales"][table][..., None]
    return x.transpose(2, 3).flatten(1, 2)[:, :s["max_len"]]


def _plain_attend(s):
    H, G, D = s["case"]["H"], s["case"]["G"], s["case"]["D"]
    q, starts, lens = s["q"], s["starts"].long(), s["lengths"].long()
    news = starts[1:] - starts[:-1]
    i = torch.arange(s["max_new"], device="cuda")
    there = i[None, :] < news[:, None]                   # [B, new]
    rows = torch.where(there, starts[:-1, None] + i[None, :], 0)
    B, n = rows.shape
    qp = q[rows].float().view(B, n, G, H // G, D).permute(0, 2, 3, 1, 4).reshape(B, G, -1, D)
    k, v = (_plain_gather(s, name).transpose(1, 2) for name in ("k", "v"))   # [B, G, keys, D]
    score = (qp @ k.transpose(2, 3)) * D ** -0.5         # [B, G, heads * new, keys]
    last = lens[:, None] - news[:, None] + i[None, :]    # a token's own position
    j = torch.arange(s["max_len"], device="cuda")
    seen = (j[None, None, :] <= last[:, :, None]) & (j < lens[:, None, None])
    seen = seen[:, None, None].expand(B, G, H // G, n, -1).reshape(score.shape)
    score = score.masked_fill(~seen, -torch.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - torch.where(top == -torch.inf, 0.0, top)).exp()
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total == 0, 1.0, total)
    o = o.view(B, G, H // G, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, H, D)
    out = torch.empty_like(q)
    out[rows[there]] = o[there].to(q.dtype)
    return out


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "gemm":
        return _plain_product(s["x"]["codes"].float(), s["x"]["scales"], s["w"],
                              _type(case["y"]))
    if op == "append":
        return _plain_append(s)
    if op == "attend":
        return _plain_attend(s)
    x = s["X"].float()
    if s["c"] is not None:
        x = x * s["c"]
    q, d = _plain_rows(x)
    if op == "rows":
        return {"codes": q.to(torch.int8), "scales": d}
    return _plain_product(q, d, s["w"], _type(case["y"]))


# ------------------------------------------------------------------------ the library's
def _library(s):
    import calibration_free_dual_b200 as dq
    case = s["case"]
    op = case["op"]
    if op == "rows":
        r = dq.row_quant(s["X"], s["c"])
        return {"codes": r["codes"], "scales": r["scales"]}
    if op == "gemm":
        return dq.w8a8_gemm(s["x"], s["w"], out_dtype=_type(case["y"]))
    if op == "linear":
        return dq.w8a8_linear(s["X"], s["w"], s["c"], out_dtype=_type(case["y"]))
    if op == "append":
        q = dq.kv_append(s["k"], s["v"], s["cache"], s["slots"], positions=s["positions"],
                         cos=s["cos"], sin=s["sin"], q=s["q"])
        return {"q": q, **s["cache"]}
    return dq.paged_attention(s["q"], s["cache"], s["table"], s["lengths"],
                              q_starts=s["starts"], max_q=s["max_new"], max_len=s["max_len"])


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------------------ 64 bits
def _f32(x):
    """One binary32 operation: its exact or 53-bit result, rounded (no double rounding can
    show: 53 >= 2 * 24 + 2)."""
    return x.float().double()


def _exact_rows(x):
    a = x.abs().amax(-1, keepdim=True)
    d = _f32(a / Q_MAX).clamp(min=TINY)
    q = _f32(x * _f32(1.0 / d)).round().clamp(-Q_MAX, Q_MAX)
    return torch.where(a == 0, 0.0, q), torch.where(a == 0, 0.0, d)[..., 0]


def _exact_turn(x, cos, sin):
    h = x.shape[-1] // 2
    y = torch.empty_like(x)
    y[..., :h] = _f32(_f32(x[..., :h] * cos) - _f32(x[..., h:] * sin))
    y[..., h:] = _f32(_f32(x[..., h:] * cos) + _f32(x[..., :h] * sin))
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rows", "linear"):
        x = s["X"].double()
        if s["c"] is not None:
            x = _f32(x * s["c"].double())
        q, d = _exact_rows(x)
        if op == "rows":
            return {"codes": None, "scales": d}
    if op in ("gemm", "linear"):
        if op == "gemm":
            q, d = s["x"]["codes"].double(), s["x"]["scales"].double()
        return torch.einsum("tk,nk->tn", q, s["w"]["codes"].double()) * d[:, None] \
            * s["w"]["scales"].double()[None, :]
    if op == "append":
        pos = s["positions"].long()
        cos, sin = (s[n].double()[pos][:, None] for n in ("cos", "sin"))
        q = _exact_turn(s["q"].double(), cos, sin)
        out = {"q": q}
        for name, x in (("k", _exact_turn(s["k"].double(), cos, sin)), ("v", s["v"].double())):
            coded = case["cache"] == "int8"
            out[name] = None if coded else s["cache"][name].double()
            if coded:
                out[name + "_scales"] = s["cache"][name + "_scales"].double()
                x = _exact_rows(x)[1]
            kept = torch.nonzero(s["slots"] >= 0)[:, 0]
            to = s["slots"][kept]
            out[name + ("_scales" if coded else "")][
                torch.div(to, case["page"], rounding_mode="floor"), :, to % case["page"]] = x[kept]
        return out
    # attention: one sequence and one key head at a time, in pieces of the new tokens
    H, G, D = case["H"], case["G"], case["D"]
    news, lens = _lengths(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, m) in enumerate(zip(news, lens)):
        pages = s["table"][b, :-(-m // case["page"])].long()
        kv = []
        for name in ("k", "v"):
            x = s["cache"][name][pages].double()
            if case["cache"] == "int8":
                x = x * s["cache"][name + "_scales"][pages].double()[..., None]
            kv.append(x.permute(1, 0, 2, 3).reshape(G, -1, D)[:, :m])
        for g in range(G):
            for lo in range(0, n, 256):
                hi = min(n, lo + 256)
                q = s["q"][at + lo:at + hi, g * (H // G):(g + 1) * (H // G)].double()
                z = torch.einsum("nhd,kd->nhk", q, kv[0][g]) / math.sqrt(D)
                own_pos = m - n + torch.arange(lo, hi, device="cuda")
                hidden = torch.arange(m, device="cuda")[None, :] > own_pos[:, None]
                z = z.masked_fill(hidden[:, None, :], -math.inf)
                out[at + lo:at + hi, g * (H // G):(g + 1) * (H // G)] = torch.einsum(
                    "nhk,kd->nhd", torch.softmax(z, -1), kv[1][g])
        at += n
    return out
