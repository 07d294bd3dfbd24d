"""The attention-layer operators of the library, as a program meets them.

Three operators make an attention layer next to the convolutions: `linear` (matrix product with bias, activation and
residual), `rope` (norms of queries and keys with the position rotation, keys and values stored to cache rows) and
`attention` (capped or distance-biased scores under length, causal, window, prefix and document masks).  A case names
one call.  `run` computes it from elementary torch operations in 32 bits, or, where `own` is true, through the library;
`exact` computes it in 64 bits.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases --

def _linear(name, rows, k, n, dtype, act="none", bias=False, residual=False):
    return {"name": name, "op": "linear", "rows": rows, "k": k, "n": n, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual}


def _rope(name, tokens, heads_q, heads_kv, head_dim, rotary_dim, dtype, layout="half", norm=True, scaling="none",
          factor=1.0, original_len=0, last=0, cache_rows=0):
    return {"name": name, "op": "rope", "tokens": tokens, "heads_q": heads_q, "heads_kv": heads_kv,
            "head_dim": head_dim, "rotary_dim": rotary_dim, "dtype": dtype, "layout": layout, "norm": norm,
            "scaling": scaling, "factor": factor, "original_len": original_len, "last": last,
            "cache_rows": cache_rows}


def _attention(name, batch, q_len, kv_len, heads_q, heads_kv, head_dim, dtype, causal=True, window=0, softcap=0.0,
               slopes=False, prefix=0, docs=0, ragged=False):
    return {"name": name, "op": "attention", "batch": batch, "q_len": q_len, "kv_len": kv_len, "heads_q": heads_q,
            "heads_kv": heads_kv, "head_dim": head_dim, "dtype": dtype, "causal": causal, "window": window,
            "softcap": softcap, "slopes": slopes, "prefix": prefix, "docs": docs, "ragged": ragged}


def listed():
    return [
        # One token through a small projection: nothing but latency.
        _linear("linear token", 1, 1024, 1536, "bf16", residual=True),
        # A step of 24 sequences through the wide projection of an MLP: the weights' bytes.
        _linear("linear batch", 24, 4096, 11264, "bf16", act="silu", bias=True),
        # Image patches of a batch, odd sizes, fp32 as the convolutions' default type.
        _linear("linear patches f32", 1571, 770, 2309, "f32", act="gelu", bias=True),
        # A long prompt through a large projection that adds to the residual stream.
        _linear("linear prompt", 8192, 4096, 8192, "bf16", bias=True, residual=True),
        # One new token of each of 32 sequences at far positions, keys and values into the cache.
        _rope("rope token", 32, 32, 8, 128, 128, "bf16", scaling="yarn", factor=16.0, original_len=8192, last=131071,
              cache_rows=8192),
        # A prompt, interleaved pairs, half of each head rotated.
        _rope("rope prompt", 16384, 32, 8, 128, 64, "bf16", layout="interleaved", last=16383),
        # A ragged number of tokens, small fp32 heads, rotated in part, linear scaling.
        _rope("rope odd f32", 1237, 6, 6, 80, 40, "f32", scaling="linear", factor=4.0, last=20000),
        # A serving step: 16 sequences of different lengths, capped scores.
        _attention("attention token", 16, 1, 4096, 32, 8, 128, "bf16", softcap=50.0, ragged=True),
        # One token over one long cache, distance bias.
        _attention("attention long cache", 1, 1, 131071, 32, 4, 128, "bf16", slopes=True),
        # A long prompt, capped scores.
        _attention("attention prompt", 1, 8192, 8192, 16, 4, 128, "bf16", softcap=30.0),
        # Documents packed into one sequence, distance bias, smaller heads.
        _attention("attention documents", 1, 6007, 6007, 12, 12, 64, "bf16", slopes=True, docs=17),
        # A batch whose prefix (an image, an instruction) is seen by all of its rows, fp32, ragged.
        _attention("attention prefix f32", 3, 517, 517, 8, 2, 96, "f32", prefix=130, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c = _draw(rng)
    del c["name"]
    return c


def _draw(rng):
    op = rng.choice(("linear", "rope", "attention", "attention"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "linear":
        while True:
            rows, k, n = _log(rng, 1, 8192), _log(rng, 64, 8192), _log(rng, 64, 11264)
            if rng.random() < 0.6:
                k, n = -(-k // 64) * 64, -(-n // 64) * 64
            if rows * k * n <= 8192 * 4096 * 8192:
                break
        return _linear("", rows, k, n, dtype, rng.choice(("none", "relu", "silu", "gelu", "gelu_tanh")),
                       rng.random() < 0.5, rng.random() < 0.5)
    if op == "rope":
        heads_kv = rng.choice((1, 2, 4, 6, 8))
        head_dim = rng.choice((32, 64, 80, 96, 128, 256))
        rotary = rng.choice((head_dim, head_dim, head_dim // 2, 24))
        heads_q = heads_kv * rng.choice((1, 2, 4, 8))
        tokens = _log(rng, 1, max(1, 16384 * 48 * 128 // ((heads_q + 2 * heads_kv) * head_dim)))
        tokens = min(tokens, 16384)
        scaling = rng.choice(("none", "linear", "yarn"))
        return _rope("", tokens, heads_q, heads_kv, head_dim, rotary, dtype, rng.choice(("half", "interleaved")),
                     rng.random() < 0.7, scaling, 1.0 if scaling == "none" else rng.choice((2.0, 4.0, 16.0)),
                     rng.choice((2048, 8192)), _log(rng, tokens, 200000),
                     0 if rng.random() < 0.5 else tokens + rng.randrange(1, 4096))
    while True:
        heads_kv = rng.choice((1, 2, 4, 8, 12))
        heads_q = heads_kv * rng.choice((1, 1, 2, 4, 8))
        batch = _log(rng, 1, 32)
        kv_len = _log(rng, 1, 131071)
        q_len = rng.choice((1, 1, rng.randrange(1, 9), _log(rng, 1, 512), kv_len, kv_len))
        head_dim = rng.choice((32, 64, 64, 96, 128, 128, 256))
        q_len = min(q_len, kv_len)
        pairs = batch * heads_q * q_len * kv_len
        cache = batch * heads_kv * kv_len * head_dim
        if pairs * head_dim <= 16 * 8192 * 8192 * 128 // (1 if dtype == "bf16" else 8) and pairs <= 16 * 8192 * 8192 \
                and cache <= 131071 * 4 * 128:
            break
    causal = rng.random() < 0.7
    kind = rng.choice(("none", "none", "prefix", "docs", "window"))
    return _attention("", batch, q_len, kv_len, heads_q, heads_kv, head_dim, dtype, causal,
                      rng.randrange(1, kv_len + 1) if kind == "window" else 0, rng.choice((0.0, 20.0, 50.0)),
                      rng.random() < 0.4, rng.randrange(0, kv_len + 1) if kind == "prefix" else 0,
                      rng.randrange(1, 20) if kind == "docs" else 0, rng.random() < 0.5)


# ----------------------------------------------------------------- inputs --

def _lengths(case):
    """(query, key) lengths of each sequence: whole, or spread over the upper three quarters."""
    b, lq, lk = case["batch"], case["q_len"], case["kv_len"]
    if not case["ragged"]:
        return [lq] * b, [lk] * b
    r = random.Random("%d %d %d" % (b, lq, lk))
    kv = [lk] + [r.randrange(max(1, lk // 4), lk + 1) for _ in range(b - 1)]
    q = [min(n, lq) if lq < lk else n for n in kv]
    return q, kv


def _offsets(case):
    """Borders of each sequence's documents, [batch][docs + 1]: of all sizes, the last one at the key length."""
    got = []
    for i, n in enumerate(_lengths(case)[1]):
        r = random.Random("%d %d %d" % (i, n, case["docs"]))
        got.append([0] + sorted(r.randrange(0, n + 1) for _ in range(case["docs"] - 1)) + [n])
    return got


def _numbers(shape, dtype, gen, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(TYPES[dtype])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, op = case["dtype"], case["op"]
    s = {"case": case}
    if op == "linear":
        m, k, n = case["rows"], case["k"], case["n"]
        s["x"] = _numbers((m, k), dt, gen)
        s["w"] = _numbers((n, k), dt, gen, k ** -0.5)
        s["bias"] = _numbers((n,), "f32", gen, 0.1) if case["bias"] else None
        s["residual"] = _numbers((m, n), dt, gen) if case["residual"] else None
        s["y"] = torch.empty((m, n), dtype=TYPES[dt], device="cuda")
    elif op == "rope":
        t, hq, hk, d = case["tokens"], case["heads_q"], case["heads_kv"], case["head_dim"]
        rows = case["cache_rows"] or t
        s["qkv"] = _numbers((t, (hq + 2 * hk) * d), dt, gen)
        s["q_gamma"] = 1 + _numbers((d,), "f32", gen, 0.1) if case["norm"] else None
        s["k_gamma"] = 1 + _numbers((d,), "f32", gen, 0.1) if case["norm"] else None
        last = case["last"]
        if case["cache_rows"]:  # tokens of different sequences, in rows of the cache that are theirs
            s["positions"] = torch.randint(0, last + 1, (t,), generator=gen, device="cuda", dtype=torch.int32)
            s["slots"] = torch.randperm(rows, generator=gen, device="cuda")[:t].to(torch.int32)
        else:
            s["positions"] = torch.arange(last - t + 1, last + 1, device="cuda", dtype=torch.int32)
            s["slots"] = None
        s["q"] = torch.empty((t, hq, d), dtype=TYPES[dt], device="cuda")
        s["k"] = torch.zeros((rows, hk, d), dtype=TYPES[dt], device="cuda")
        s["v"] = torch.zeros((rows, hk, d), dtype=TYPES[dt], device="cuda")
    else:
        b, hq, hk, d = case["batch"], case["heads_q"], case["heads_kv"], case["head_dim"]
        q_lens, kv_lens = _lengths(case)
        # Scores spread over a few units, so that a cap and a softmax have something to do.
        s["q"] = _numbers((b, case["q_len"], hq, d), dt, gen, 2.5)
        s["k"] = _numbers((b, case["kv_len"], hk, d), dt, gen)
        s["v"] = _numbers((b, case["kv_len"], hk, d), dt, gen)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        s["q_lens"] = ints(q_lens) if case["ragged"] else None
        s["kv_lens"] = ints(kv_lens) if case["ragged"] else None
        s["prefix_lens"] = ints([min(case["prefix"] + i, n) for i, n in enumerate(kv_lens)]) if case["prefix"] else None
        s["doc_offsets"] = ints(_offsets(case)) if case["docs"] else None
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda", dtype=torch.float32) / hq) \
            if case["slopes"] else None
        s["out"] = torch.empty((b, case["q_len"], hq, d), dtype=TYPES[dt], device="cuda")
    if own:
        _plan(s)
    return s


def _plan(s):
    """The descriptor, and the workspace where there is one, that a program keeps for its calls."""
    import convolution_conv2d_forward_amd as cc
    c = s["case"]
    if c["op"] == "linear":
        s["desc"] = cc.linear_desc_create(cc.make_linear_params(
            c["k"], c["n"], has_bias=c["bias"], act=c["act"], has_residual=c["residual"], dtype=c["dtype"]))
    elif c["op"] == "rope":
        s["desc"] = cc.qk_rope_desc_create(cc.make_qk_rope_params(
            c["heads_q"], c["heads_kv"], c["head_dim"], rotary_dim=c["rotary_dim"], layout=c["layout"],
            has_norm=c["norm"], scaling=c["scaling"], factor=c["factor"], original_len=c["original_len"],
            dtype=c["dtype"]))
    else:
        s["desc"] = cc.attention_desc_create(cc.make_attention_params(
            c["heads_q"], c["heads_kv"], c["head_dim"], causal=c["causal"], window=c["window"],
            softcap=c["softcap"], has_slopes=c["slopes"], q_strides=s["q"].stride()[:3], k_strides=s["k"].stride()[:3],
            v_strides=s["v"].stride()[:3], out_strides=s["out"].stride()[:3], dtype=c["dtype"]))
        n = cc.attention_workspace_bytes(s["desc"], c["batch"], c["q_len"], c["kv_len"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


# -------------------------------------------------------------------- run --

def run(s):
    op = s["case"]["op"]
    if own:
        return _call(s)
    return _plain_linear(s) if op == "linear" else _plain_rope(s) if op == "rope" else _plain_attention(s)


def _call(s):
    import convolution_conv2d_forward_amd as cc
    op = s["case"]["op"]
    if op == "linear":
        cc.linear_forward(s["desc"], s["x"], s["w"], s["bias"], s["residual"], s["y"])
        return s["y"]
    if op == "rope":
        cc.qk_rope_forward(s["desc"], s["qkv"], s["q_gamma"], s["k_gamma"], s["positions"], s["slots"], s["q"],
                           s["k"], s["v"])
        return s["q"], s["k"], s["v"]
    cc.attention_forward(s["desc"], s["q"], s["k"], s["v"], s["out"], q_lens=s["q_lens"], kv_lens=s["kv_lens"],
                         prefix_lens=s["prefix_lens"], doc_offsets=s["doc_offsets"], slopes=s["slopes"],
                         workspace=s["workspace"])
    return s["out"]


def _plain_linear(s):
    c = s["case"]
    y = torch.matmul(s["x"].float(), s["w"].float().t())
    if c["bias"]:
        y = y + s["bias"]
    if c["act"] == "relu":
        y = torch.clamp(y, min=0)
    elif c["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif c["act"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif c["act"] == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if c["residual"]:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


THETA, EPS, FAST, SLOW = 10000.0, 1e-6, 32.0, 1.0


def _plain_frequencies(c):
    """Angle a position of each pair, in 64 bits, and the factor on the rotated values."""
    r = c["rotary_dim"]
    i = torch.arange(r // 2, device="cuda", dtype=torch.float64)
    f = THETA ** (-2 * i / r)
    if c["scaling"] == "linear":
        return f / c["factor"], 1.0
    if c["scaling"] == "yarn":
        turn = lambda n: r * math.log(c["original_len"] / (2 * math.pi * n)) / (2 * math.log(THETA))  # noqa: E731
        lo, hi = max(math.floor(turn(FAST)), 0), min(math.ceil(turn(SLOW)), r - 1)
        ramp = torch.clamp((i - lo) / max(hi - lo, 0.001), 0, 1)
        return f * (1 - ramp) + f / c["factor"] * ramp, 0.1 * math.log(c["factor"]) + 1
    return f, 1.0


def _plain_rotate(x, gamma, cos, sin, c):
    r = c["rotary_dim"]
    x = x.float()
    if c["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma
    y = x.clone()
    if c["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_rope(s):
    c = s["case"]
    t, hq, hk, d = c["tokens"], c["heads_q"], c["heads_kv"], c["head_dim"]
    f, factor = _plain_frequencies(c)
    angle = s["positions"].double()[:, None, None] * f
    cos, sin = (torch.cos(angle) * factor).float(), (torch.sin(angle) * factor).float()
    dt = s["qkv"].dtype
    x = s["qkv"].view(t, hq + 2 * hk, d)
    q = _plain_rotate(x[:, :hq], s["q_gamma"], cos, sin, c).to(dt)
    k = _plain_rotate(x[:, hq:hq + hk], s["k_gamma"], cos, sin, c).to(dt)
    if s["slots"] is None:
        return q, k, x[:, hq + hk:].clone()
    rows = s["slots"].long()
    s["k"][rows], s["v"][rows] = k, x[:, hq + hk:]
    return q, s["k"], s["v"]


def _plain_allowed(s, at, j, kv, b):
    """Which keys j ([1, 1, Lk]) the queries at positions `at` ([B, Lq, 1]) see; kv: the sequences' lengths."""
    c = s["case"]
    see = (j < kv) & (at >= 0 if c["causal"] or c["docs"] else at == at)
    if c["causal"]:
        before = j <= at
        if c["prefix"]:
            before = before | (j < s["prefix_lens"].view(b, 1, 1))
            see = j < kv
        see = see & before
    if c["window"]:
        see = see & ((at - j).abs() < c["window"])
    if c["docs"]:
        border = s["doc_offsets"].view(b, 1, 1, -1)
        doc_k = (j.unsqueeze(-1) >= border).sum(-1)
        doc_q = (at.unsqueeze(-1) >= border).sum(-1)
        see = see & (doc_k == doc_q)
    return see


def _plain_attention(s):
    c = s["case"]
    b, lq, lk, hq, hk, d = c["batch"], c["q_len"], c["kv_len"], c["heads_q"], c["heads_kv"], c["head_dim"]
    g = hq // hk
    q = s["q"].float().view(b, lq, hk, g, d).permute(0, 2, 3, 1, 4).reshape(b, hk, g * lq, d)
    k = s["k"].float().permute(0, 2, 3, 1).contiguous()
    v = s["v"].float().permute(0, 2, 1, 3).contiguous()
    dev = q.device
    nq = torch.full((b,), lq, device=dev) if s["q_lens"] is None else s["q_lens"].long()
    nk = torch.full((b,), lk, device=dev) if s["kv_lens"] is None else s["kv_lens"].long()
    i, j = torch.arange(lq, device=dev).view(1, lq, 1), torch.arange(lk, device=dev).view(1, 1, lk)
    nq, nk = nq.view(b, 1, 1), nk.view(b, 1, 1)
    at = nk - nq + i
    see = _plain_allowed(s, at, j, nk, b) & (i < nq)
    p = torch.matmul(q, k).mul_(d ** -0.5).view(b, hk, g, lq, lk)
    if c["softcap"]:
        p = p.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    if c["slopes"]:
        p.addcmul_(s["slopes"].view(1, hk, g, 1, 1), (at - j).abs().float().view(b, 1, 1, lq, lk), value=-1)
    p.masked_fill_(~see.view(b, 1, 1, lq, lk), -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(b, hk, g * lq, lk), v).view(b, hk, g, lq, d)
    out = out / torch.where(total == 0, torch.ones_like(total), total)
    return out.permute(0, 3, 1, 2, 4).reshape(b, lq, hq, d).to(s["q"].dtype)


# ------------------------------------------------------------------- work --

def _pairs(case):
    """Allowed (query, key) pairs of one head over the batch."""
    total = 0
    borders = _offsets(case) if case["docs"] else None
    for b, (nq, nk) in enumerate(zip(*_lengths(case))):
        at = torch.arange(nk - nq, nk)
        lo, hi = torch.zeros_like(at), torch.full_like(at, nk)
        if case["docs"]:
            edges = torch.tensor(borders[b])
            doc = torch.searchsorted(edges, at, right=True)
            lo, hi = edges[(doc - 1).clamp(min=0)], edges[doc.clamp(max=len(edges) - 1)]
        if case["window"]:
            lo, hi = torch.maximum(lo, at - case["window"] + 1), torch.minimum(hi, at + case["window"])
        if case["causal"]:
            seen = min(case["prefix"] + b, nk) if case["prefix"] else 0
            hi = torch.minimum(hi, (at + 1).clamp(min=seen))
        total += int((hi - lo).clamp(min=0).sum())
    return total


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "linear":
        m, k, n = case["rows"], case["k"], case["n"]
        return {"bytes": size * (m * k + n * k + m * n * (2 if case["residual"] else 1)) + (4 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    if case["op"] == "rope":
        t, hq, hk, d = case["tokens"], case["heads_q"], case["heads_kv"], case["head_dim"]
        return {"bytes": 2 * size * t * (hq + 2 * hk) * d + 4 * t, "flops": t * (hq + hk) * (6 * case["rotary_dim"] // 2 + 4 * d)}
    q_lens, kv_lens = _lengths(case)
    hq, hk, d = case["heads_q"], case["heads_kv"], case["head_dim"]
    rows = case["batch"] * case["q_len"]
    return {"bytes": size * d * (hq * (sum(q_lens) + rows) + 2 * hk * sum(kv_lens)), "flops": 4 * d * hq * _pairs(case)}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _exact_linear(s, case)
    return _exact_rope(s, case) if case["op"] == "rope" else _exact_attention(s, case)


def _exact_linear(s, c):
    y = s["x"].double() @ s["w"].double().T
    if c["bias"]:
        y += s["bias"].double()
    if c["act"] == "relu":
        y = torch.where(y > 0, y, torch.zeros_like(y))
    elif c["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif c["act"] == "gelu":
        y = y * 0.5 * torch.erfc(-y / 2 ** 0.5)
    elif c["act"] == "gelu_tanh":
        y = y / (1 + torch.exp(-2 * (2 / math.pi) ** 0.5 * (y + 0.044715 * y ** 3)))
    return y + s["residual"].double() if c["residual"] else y


def _exact_rope(s, c):
    t, hq, hk, d, r = c["tokens"], c["heads_q"], c["heads_kv"], c["head_dim"], c["rotary_dim"]
    angles, factor = [], 1.0
    for i in range(r // 2):
        f = math.exp(-2.0 * i / r * math.log(THETA))
        if c["scaling"] == "linear":
            f /= c["factor"]
        elif c["scaling"] == "yarn":
            per = r / (2 * math.log(THETA))
            first = max(0, math.floor(per * math.log(c["original_len"] / (FAST * 2 * math.pi))))
            last = min(r - 1, math.ceil(per * math.log(c["original_len"] / (SLOW * 2 * math.pi))))
            share = min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
            f = f * (1 - share) + f * share / c["factor"]
            factor = 1 + math.log(c["factor"]) / 10
        angles.append(f)
    turn = torch.polar(torch.full((t, r // 2), factor, dtype=torch.float64, device="cuda"),
                       s["positions"].double()[:, None] * torch.tensor(angles, dtype=torch.float64, device="cuda"))

    def head(x, gamma):
        x = x.double()
        if gamma is not None:
            x = x / (x.square().sum(-1, keepdim=True) / d + EPS).sqrt() * gamma.double()
        part = x[..., :r].unflatten(-1, (2, r // 2) if c["layout"] == "half" else (r // 2, 2))
        part = part.transpose(-1, -2) if c["layout"] == "half" else part
        part = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn[:, None])
        part = part.transpose(-1, -2) if c["layout"] == "half" else part
        return torch.cat((part.flatten(-2), x[..., r:]), -1)

    q, k, v = s["qkv"].view(t, -1, d).split((hq, hk, hk), 1)
    q, k, v = head(q, s["q_gamma"]), head(k, s["k_gamma"]), v.double()
    if s["slots"] is None:
        return q, k, v
    full = [torch.zeros((c["cache_rows"], hk, d), dtype=torch.float64, device="cuda") for _ in "kv"]
    for rows, x in zip(full, (k, v)):
        rows.index_copy_(0, s["slots"].long(), x)
    return q, full[0], full[1]


def _exact_attention(s, c):
    b, lq, hq, d = s["q"].shape
    group = hq // c["heads_kv"]
    out = torch.zeros((b, lq, hq, d), dtype=torch.float64, device="cuda")
    q_lens, kv_lens = _lengths(c)
    borders = _offsets(c) if c["docs"] else None
    slopes = s["slopes"].tolist() if c["slopes"] else None
    for n in range(b):
        nq, nk = q_lens[n], kv_lens[n]
        dist = torch.arange(nk - nq, nk, device="cuda")[:, None] - torch.arange(nk, device="cuda")[None, :]
        seen = torch.ones((nq, nk), dtype=torch.bool, device="cuda")
        if c["causal"]:
            seen = torch.tril(seen, diagonal=nk - nq)
            if c["prefix"]:
                seen[:, :min(c["prefix"] + n, nk)] = True
        if c["window"]:
            seen &= (dist < c["window"]) & (dist > -c["window"])
        if c["docs"]:
            same = torch.zeros_like(seen)
            for first, end in zip(borders[n], borders[n][1:]):
                same[max(0, first - (nk - nq)):max(0, end - (nk - nq)), first:end] = True
            seen &= same
        for h in range(hq):
            a = s["q"][n, :nq, h].double() @ s["k"][n, :nk, h // group].double().T / d ** 0.5
            if c["softcap"]:
                a = c["softcap"] * torch.tanh(a / c["softcap"])
            if slopes:
                a = a - slopes[h] * dist.abs()
            a = torch.where(seen, a, torch.full_like(a, -math.inf))
            a = torch.exp(a - torch.logsumexp(a, 1, keepdim=True))
            out[n, :nq, h] = torch.nan_to_num(a) @ s["v"][n, :nk, h // group].double()
    return out
