"""The operators of a decoder layer over a paged cache, as a serving program meets them.

`store` writes the keys and values of new tokens to pages, quantised to 8 bits with a power of two a token and head;
`load` reads sequences back from their pages; `attend` is softmax attention of each sequence's new tokens (a chunk of a
prompt, single tokens, both in one batch) over its pages, with a sliding window and first tokens that stay visible;
`norm` is the norm behind a block, its gate and residual scale, and the norm before the next one.  A case names one
call.  `run` computes it from elementary torch operations in 32 bits, or, where `own` is true, through the library;
`exact` computes it in 64 bits.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZES = {"f32": 4, "bf16": 2, "e4m3": 1}


# ------------------------------------------------------------------ cases --

def _store(name, tokens, heads_kv, head_dim, page_size, pages, dtype, cache):
    return {"name": name, "op": "store", "tokens": tokens, "heads_kv": heads_kv, "head_dim": head_dim,
            "page_size": page_size, "pages": pages, "dtype": dtype, "cache": cache}


def _load(name, batch, context, heads_kv, head_dim, page_size, dtype, cache, ragged=True):
    return {"name": name, "op": "load", "batch": batch, "context": context, "heads_kv": heads_kv,
            "head_dim": head_dim, "page_size": page_size, "dtype": dtype, "cache": cache, "ragged": ragged}


def _attend(name, batch, chunk, context, heads_q, heads_kv, head_dim, page_size, dtype, cache, window=0, sinks=0,
            softcap=0.0, ragged=False, chunks=0):
    """`chunks` > 0: so many sequences bring `chunk` new tokens, the others one."""
    return {"name": name, "op": "attend", "batch": batch, "chunk": chunk, "context": context, "heads_q": heads_q,
            "heads_kv": heads_kv, "head_dim": head_dim, "page_size": page_size, "dtype": dtype, "cache": cache,
            "window": window, "sinks": sinks, "softcap": softcap, "ragged": ragged, "chunks": chunks}


def _norm(name, rows, width, dtype, post="rms", pre="rms", gate_rows=0, residual_scale=1.0, block_scale=1.0):
    """gate_rows: rows that share a row of the gate; 0: one row for all, -1: no gate."""
    return {"name": name, "op": "norm", "rows": rows, "width": width, "dtype": dtype, "post": post, "pre": pre,
            "gate_rows": gate_rows, "residual_scale": residual_scale, "block_scale": block_scale}


def listed():
    return [
        # A serving step of 64 sequences: one new token of each into its page.  Nothing but latency.
        _store("store token", 64, 8, 128, 16, 1024, "bf16", "e4m3"),
        # A long prompt's keys and values.
        _store("store prompt", 16384, 8, 128, 64, 320, "bf16", "e4m3"),
        # Four cached prefixes read back for a batch that attends to them as dense tensors.
        _load("load prefix", 4, 8192, 8, 128, 16, "bf16", "e4m3"),
        # A small fp32 cache with pages of 24 tokens, moved.
        _load("load odd f32", 3, 1531, 6, 80, 24, "f32", "f32"),
        # A serving step: 32 sequences of different lengths, one token each, 8-bit cache.
        _attend("attend token", 32, 1, 8192, 32, 8, 128, 16, "bf16", "e4m3", ragged=True),
        # One token over one long 16-bit cache.
        _attend("attend long", 1, 1, 131071, 32, 4, 128, 64, "bf16", "bf16"),
        # A chunk of a long prompt over all that came before it.
        _attend("attend chunk", 1, 2048, 32768, 16, 4, 128, 64, "bf16", "bf16"),
        # A step that carries two chunks of prompts among single tokens, capped scores, 8-bit cache.
        _attend("attend mixed", 16, 256, 4096, 16, 4, 128, 32, "bf16", "e4m3", softcap=30.0, ragged=True, chunks=2),
        # Chunks under a sliding window with first tokens that stay visible, smaller heads, odd lengths.
        _attend("attend window", 2, 1500, 20001, 12, 12, 64, 48, "bf16", "bf16", window=1024, sinks=4),
        # Ragged fp32 sequences, a few drafted tokens to a short chunk, pages of 20.
        _attend("attend odd f32", 3, 77, 1537, 8, 2, 96, 20, "f32", "f32", window=500, sinks=3, ragged=True),
        # A serving step's rows between two blocks.
        _norm("norm token", 24, 4096, "bf16"),
        # A batch of four prompts, a gate row for each, scaled residuals.
        _norm("norm prompt", 8192, 4096, "bf16", "layer", "layer", 2048, 0.75, 0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c = _draw(rng)
    del c["name"]
    return c


def _draw(rng):
    op = rng.choice(("store", "load", "attend", "attend", "attend", "norm"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    cache = rng.choice(("e4m3", dtype))
    heads_kv = rng.choice((1, 2, 4, 6, 8, 12))
    head_dim = rng.choice((32, 64, 64, 80, 96, 128, 128, 256))
    page_size = rng.choice((1, 8, 16, 16, 20, 32, 48, 64, 128, 256))
    most = 131071 * 4 * 128   # elements of a cache's keys
    if op == "store":
        tokens = _log(rng, 1, min(16384, 16384 * 8 * 128 // (heads_kv * head_dim)))
        pages = -(-tokens // page_size) + rng.randrange(1, 40)
        return _store("", tokens, heads_kv, head_dim, page_size, pages, dtype, cache)
    if op == "load":
        batch = _log(rng, 1, 32)
        context = _log(rng, 1, max(1, min(32768, most // 2 // (batch * heads_kv * head_dim))))
        return _load("", batch, context, heads_kv, head_dim, page_size, dtype, cache, rng.random() < 0.7)
    if op == "norm":
        width = rng.choice((_log(rng, 16, 16384), 8 * _log(rng, 8, 2048)))
        rows = _log(rng, 1, max(1, min(16384, 8192 * 4096 // width)))
        kinds = rng.choice((("rms", "rms"), ("none", "rms"), ("none", "layer"), ("rms", "none"), ("layer", "layer")))
        return _norm("", rows, width, dtype, *kinds, rng.choice((-1, 0, 0, rng.randrange(1, rows + 1))),
                     rng.choice((1.0, 0.7)), rng.choice((1.0, 0.3)))
    while True:
        heads_q = heads_kv * rng.choice((1, 1, 2, 4, 8))
        batch = _log(rng, 1, 48)
        context = _log(rng, 1, 131071)
        chunk = min(context, rng.choice((1, 1, rng.randrange(1, 9), _log(rng, 1, 512), _log(rng, 64, 4096))))
        pairs = batch * heads_q * chunk * context
        if pairs * (1 if dtype == "bf16" else 8) <= 16 * 2048 * 32768 and \
                pairs * head_dim * (1 if dtype == "bf16" else 8) <= 16 * 2048 * 32768 * 128 and \
                batch * heads_kv * context * head_dim <= most:
            break
    window = rng.choice((0, 0, _log(rng, 1, context)))
    return _attend("", batch, chunk, context, heads_q, heads_kv, head_dim, page_size, dtype, cache, window,
                   rng.randrange(0, 20) if window else 0, rng.choice((0.0, 0.0, 20.0, 50.0)), rng.random() < 0.6,
                   rng.randrange(1, batch + 1) if chunk > 1 and rng.random() < 0.4 else 0)


# ----------------------------------------------------------------- inputs --

EPS = 1e-6


def _lengths(case):
    """(new, all) tokens of each sequence: whole, or spread over the upper three quarters."""
    b, context = case["batch"], case["context"]
    kv = [context] * b
    if case["ragged"]:
        r = random.Random("%d %d" % (b, context))
        kv = [context] + [r.randrange(max(1, context // 4), context + 1) for _ in range(b - 1)]
    if case["op"] == "load":
        return None, kv
    few = case["chunks"] or b
    return [min(n, case["chunk"] if i < few else 1) for i, n in enumerate(kv)], kv


def _pages(case):
    """Pages in the cache, and pages that the longest sequence takes."""
    ps = case["page_size"]
    return sum(-(-n // ps) for n in _lengths(case)[1]) + 3, -(-case["context"] // ps)


def _numbers(shape, dtype, gen, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(TYPES[dtype])


def _keys(shape, dtype, gen):
    """Keys and values as projections give them: heads of different size, a channel that stands out."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    x *= torch.exp(0.3 * torch.randn(shape[:-1], generator=gen, device="cuda")).unsqueeze(-1)
    x[..., 3] *= 6.0
    return x.to(TYPES[dtype])


def _cache(case, pages, gen, filled):
    """k and v pages [pages, page_size, heads, dim] of the cache's type, with the scales' exponents if it has any."""
    shape = (pages, case["page_size"], case["heads_kv"], case["head_dim"])
    got = {}
    for n in "kv":
        if not filled:
            x, e = torch.zeros(shape, device="cuda", dtype=TYPES[case["cache"]]), None
            if case["cache"] == "e4m3":
                e = torch.zeros(shape[:-1], device="cuda", dtype=torch.uint8)
        else:
            x, e = _keys(shape, case["dtype"], gen), None
            if case["cache"] == "e4m3":
                x, e = _quantise(x)
        got[n + "_pages"], got[n + "_scales"] = x, e
    return got


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, op = case["dtype"], case["op"]
    s = {"case": case}
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if op == "store":
        t, h, d = case["tokens"], case["heads_kv"], case["head_dim"]
        # Keys come rotated, in a buffer of their own; values lie in the projection's rows, behind queries and keys.
        s["k"] = _keys((t, h, d), dt, gen)
        s["v"] = _keys((t, 3 * h, d), dt, gen)[:, 2 * h:]
        slots = case["pages"] * case["page_size"]
        s["slots"] = torch.randperm(slots, generator=gen, device="cuda")[:t].to(torch.int32)
        s.update(_cache(case, case["pages"], gen, False))
    elif op in ("load", "attend"):
        q_lens, kv_lens = _lengths(case)
        pages, longest = _pages(case)
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        need = ints([-(-n // case["page_size"]) for n in kv_lens])
        column = torch.arange(longest, device="cuda")
        at = (need.cumsum(0) - need)[:, None] + column
        s["page_table"] = torch.where(column < need[:, None], order[at.clamp(max=pages - 1)], -1).to(torch.int32)
        s["kv_lens"] = ints(kv_lens)
        s.update(_cache(case, pages, gen, True))
        b, h, d = case["batch"], case["heads_kv"], case["head_dim"]
        if op == "load":
            for n in "kv":
                s[n] = torch.zeros((b, case["context"], h, d), device="cuda", dtype=TYPES[dt])
        else:
            total = sum(q_lens)
            s["tokens"], s["longest"] = total, max(q_lens)
            s["q_offsets"] = ints([sum(q_lens[:i]) for i in range(b + 1)])
            # Scores spread over a few units, so that a cap and a softmax have something to do.
            s["q"] = _numbers((total, case["heads_q"], d), dt, gen, 1.5)
            s["out"] = torch.empty((total, case["heads_q"], d), device="cuda", dtype=TYPES[dt])
    else:
        m, d = case["rows"], case["width"]
        s["y"], s["x"] = _numbers((m, d), dt, gen, 3.0), _numbers((m, d), dt, gen)
        s["gate"] = None
        if case["gate_rows"] >= 0:
            s["gate"] = _numbers((-(-m // case["gate_rows"]) if case["gate_rows"] else 1, d), dt, gen, 0.5)
        for n in ("post", "pre"):
            s[n + "_gamma"] = 1 + _numbers((d,), "f32", gen, 0.1) if case[n] != "none" else None
            s[n + "_beta"] = _numbers((d,), "f32", gen, 0.1) if case[n] == "layer" else None
        s["residual"] = torch.empty((m, d), device="cuda", dtype=TYPES[dt])
        s["out"] = torch.empty((m, d), device="cuda", dtype=TYPES[dt]) if case["pre"] != "none" else None
    if own:
        _plan(s)
    return s


def _plan(s):
    """The descriptor, and the workspace where there is one, that a program keeps for its calls."""
    import convolution_conv2d_forward_amd as cc
    c = s["case"]
    if c["op"] == "norm":
        s["desc"] = cc.block_norm_desc_create(cc.make_block_norm_params(
            c["width"], post_norm=c["post"], pre_norm=c["pre"], has_post_beta=s["post_beta"] is not None,
            has_pre_beta=s["pre_beta"] is not None, has_gate=c["gate_rows"] >= 0, gate_rows=max(c["gate_rows"], 0),
            residual_scale=c["residual_scale"], block_scale=c["block_scale"], eps=EPS, dtype=c["dtype"]))
    elif c["op"] == "attend":
        s["desc"] = cc.paged_attention_desc_create(cc.make_paged_attention_params(
            c["heads_q"], c["heads_kv"], c["head_dim"], c["page_size"], window=c["window"], sinks=c["sinks"],
            softcap=c["softcap"], dtype=c["dtype"], cache_dtype=c["cache"]))
        n = cc.paged_attention_workspace_bytes(s["desc"], s["tokens"], c["batch"], s["page_table"].shape[1])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    else:
        strides = {"k_stride": s["k"].stride(0), "v_stride": s["v"].stride(0)} if c["op"] == "store" else {}
        s["desc"] = cc.kv_cache_desc_create(cc.make_kv_cache_params(
            c["heads_kv"], c["head_dim"], c["page_size"], dtype=c["dtype"], cache_dtype=c["cache"], **strides))


# -------------------------------------------------------------------- run --

def run(s):
    op = s["case"]["op"]
    if own:
        return _call(s)
    return {"store": _plain_store, "load": _plain_load, "attend": _plain_attend, "norm": _plain_norm}[op](s)


def _call(s):
    import convolution_conv2d_forward_amd as cc
    op = s["case"]["op"]
    if op == "store":
        cc.kv_cache_store(s["desc"], s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"], s["k_scales"],
                          s["v_scales"])
        return s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]
    if op == "load":
        cc.kv_cache_load(s["desc"], s["page_table"], s["kv_lens"], s["k_pages"], s["v_pages"], s["k_scales"],
                         s["v_scales"], s["k"], s["v"])
        return s["k"], s["v"]
    if op == "attend":
        cc.paged_attention_forward(s["desc"], s["q"], s["q_offsets"], s["kv_lens"], s["page_table"], s["k_pages"],
                                   s["v_pages"], s["k_scales"], s["v_scales"], s["out"], workspace=s["workspace"])
        return s["out"]
    cc.block_norm_forward(s["desc"], s["y"], s["x"], s["gate"], s["post_gamma"], s["post_beta"], s["pre_gamma"],
                          s["pre_beta"], s["residual"], s["out"])
    return s["residual"], s["out"]


def _power(e):
    """2^e in fp32 from a tensor of whole numbers -126 .. 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """(e4m3 codes, exponents + 127) of the rows of x: the least power of two that brings the largest to 448 at most."""
    x = x.float()
    top = x.abs().amax(-1)
    part, e = torch.frexp(top)
    e = torch.where(part > 0.875, e - 8, e - 9)   # 448 = 0.875 * 2^9
    e = torch.where(top == 0, -117, e.clamp(-117, 120))
    return (x * _power(-e).unsqueeze(-1)).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _plain_store(s):
    at = s["slots"].long()
    for n in "kv":
        x, pages, scales = s[n], s[n + "_pages"], s[n + "_scales"]
        if scales is not None:
            x, e = _quantise(x)
            scales.view(-1, scales.shape[-1])[at] = e
            x, pages = x.view(torch.uint8), pages.view(torch.uint8)
        pages.view(-1, *pages.shape[2:])[at] = x
    return s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]


def _plain_rows(s, n):
    """Keys or values of all sequences in fp32, [batch, context, heads, dim], whatever lies past their lengths."""
    c = s["case"]
    j = torch.arange(c["context"], device="cuda")
    at = s["page_table"].long()[:, j // c["page_size"]].clamp(min=0) * c["page_size"] + j % c["page_size"]
    pages, scales = s[n + "_pages"], s[n + "_scales"]
    flat = pages.view(-1, *pages.shape[2:])
    if scales is None:
        return flat[at].float()
    x = flat.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    return x * _power(scales.view(-1, scales.shape[-1])[at].to(torch.int32) - 127).unsqueeze(-1)


def _plain_load(s):
    c = s["case"]
    there = (torch.arange(c["context"], device="cuda") < s["kv_lens"][:, None])[:, :, None, None]
    for n in "kv":
        s[n].copy_(torch.where(there, _plain_rows(s, n), s[n].float()))
    return s["k"], s["v"]


def _plain_attend(s):
    c = s["case"]
    b, lq, lk, hq, hk, d = c["batch"], s["longest"], c["context"], c["heads_q"], c["heads_kv"], c["head_dim"]
    g = hq // hk
    k = _plain_rows(s, "k").permute(0, 2, 3, 1).contiguous()
    v = _plain_rows(s, "v").permute(0, 2, 1, 3).contiguous()
    off, nk = s["q_offsets"].long(), s["kv_lens"].long().view(b, 1, 1)
    i, j = torch.arange(lq, device="cuda"), torch.arange(lk, device="cuda").view(1, 1, lk)
    v.masked_fill_((j >= nk).view(b, 1, lk, 1), 0)
    # Each sequence's rows beside each other, the shorter ones' filled up.
    token = off[:-1, None] + i
    live = token < off[1:, None]
    q = s["q"].float()[token.clamp(max=s["tokens"] - 1)]
    q = q.view(b, lq, hk, g, d).permute(0, 2, 3, 1, 4).reshape(b, hk, g * lq, d)
    p = torch.matmul(q, k).mul_(d ** -0.5).view(b, hk, g, lq, lk)
    at = nk - (off[1:] - off[:-1]).view(b, 1, 1) + i.view(1, lq, 1)
    see = (j <= at) & (j < nk)
    if c["window"]:
        see = see & ((at - j < c["window"]) | (j < c["sinks"]))
    if c["softcap"]:
        p = p.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    p.masked_fill_(~see.view(b, 1, 1, lq, lk), -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(b, hk, g * lq, lk), v).view(b, hk, g, lq, d)
    out = out / torch.where(total == 0, torch.ones_like(total), total)
    out = out.permute(0, 3, 1, 2, 4).reshape(b, lq, hq, d)
    return out[live].to(s["q"].dtype)


def _plain_rule(x, kind, gamma, beta):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma
    return x if beta is None else x + beta


def _plain_norm(s):
    c = s["case"]
    u = _plain_rule(s["y"].float(), c["post"], s["post_gamma"], s["post_beta"])
    if c["gate_rows"] >= 0:
        gate = s["gate"].float()
        u = u * (gate.repeat_interleave(c["gate_rows"], 0)[:c["rows"]] if c["gate_rows"] else gate)
    r = c["residual_scale"] * s["x"].float() + c["block_scale"] * u
    out = _plain_rule(r, c["pre"], s["pre_gamma"], s["pre_beta"])
    return r.to(s["x"].dtype), out.to(s["x"].dtype) if c["pre"] != "none" else None


# ------------------------------------------------------------------- work --

def _pairs(case):
    """(seen pairs of one query head, keys that some row sees) over the batch."""
    pairs = keys = 0
    for nq, nk in zip(*_lengths(case)):
        at = torch.arange(nk - nq, nk)
        low = (at - case["window"] + 1).clamp(min=0) if case["window"] else torch.zeros_like(at)
        first = torch.minimum(low, torch.full_like(low, case["sinks"]))
        pairs += int((at + 1 - low + first).sum())
        keys += nk - int(low[0]) + int(first[0])
    return pairs, keys


def work(case):
    size, small = SIZES[case["dtype"]], SIZES[case["cache"]] if "cache" in case else 0
    if case["op"] == "norm":
        m, d = case["rows"], case["width"]
        n = m * d * (3 + (case["pre"] != "none"))
        if case["gate_rows"] >= 0:
            n += (-(-m // case["gate_rows"]) if case["gate_rows"] else 1) * d
        vectors = sum(case[k] != "none" for k in ("post", "pre")) + sum(case[k] == "layer" for k in ("post", "pre"))
        return {"bytes": size * n + 4 * d * vectors, "flops": 12 * m * d}
    h, d = case["heads_kv"], case["head_dim"]
    row = 2 * h * (d * small + (case["cache"] == "e4m3"))   # a token in the cache
    if case["op"] == "store":
        return {"bytes": case["tokens"] * (row + 2 * h * d * size + 4), "flops": 4 * case["tokens"] * h * d}
    if case["op"] == "load":
        n = sum(_lengths(case)[1])
        return {"bytes": n * (row + 2 * h * d * size), "flops": 2 * n * h * d}
    pairs, keys = _pairs(case)
    q = sum(_lengths(case)[0]) * case["heads_q"] * d
    return {"bytes": keys * row + 2 * q * size, "flops": 4 * d * case["heads_q"] * pairs}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "load": _exact_load, "attend": _exact_attend, "norm": _exact_norm}[case["op"]](s, case)


def _exact_store(s, c):
    got = []
    scales = []
    for n in "kv":
        x = s[n].double()
        if c["cache"] == "e4m3":
            top = x.abs().max(-1, keepdim=True).values
            e = torch.ceil(torch.log2(top / 448)).clamp(-117, 120)
            x = x / torch.exp2(e)
            step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
            x = torch.round(x / step) * step
            full = torch.zeros(c["pages"] * c["page_size"], c["heads_kv"], device="cuda", dtype=torch.int64)
            scales.append(full.index_copy(0, s["slots"].long(), e[..., 0].long() + 127).view(s[n + "_scales"].shape))
        full = torch.zeros((c["pages"] * c["page_size"], c["heads_kv"], c["head_dim"]), device="cuda", dtype=torch.float64)
        got.append(full.index_copy(0, s["slots"].long(), x).view(s[n + "_pages"].shape))
    return got[0], got[1], *(scales or (None, None))


def _exact_sequence(s, c, n, i, length):
    """Rows [length, heads, dim] of sequence i in 64 bits."""
    table = s["page_table"][i, :-(-length // c["page_size"])].long()
    x = s[n + "_pages"].view(torch.uint8)[table].view(s[n + "_pages"].dtype).flatten(0, 1)[:length].double()
    if c["cache"] == "e4m3":
        x = x * torch.exp2(s[n + "_scales"][table].flatten(0, 1)[:length].double() - 127).unsqueeze(-1)
    return x


def _exact_load(s, c):
    got = {n: torch.zeros(s[n].shape, device="cuda", dtype=torch.float64) for n in "kv"}
    for i, length in enumerate(_lengths(c)[1]):
        for n in "kv":
            got[n][i, :length] = _exact_sequence(s, c, n, i, length)
    return got["k"], got["v"]


def _exact_attend(s, c):
    out, group, d = [], c["heads_q"] // c["heads_kv"], c["head_dim"]
    first = 0
    for i, (nq, nk) in enumerate(zip(*_lengths(c))):
        k, v = (_exact_sequence(s, c, n, i, nk) for n in "kv")
        back = torch.arange(nk - nq, nk, device="cuda")[:, None] - torch.arange(nk, device="cuda")[None, :]
        hidden = back < 0
        if c["window"]:
            far = back >= c["window"]
            far[:, :c["sinks"]] = False
            hidden |= far
        heads = []
        for h in range(c["heads_q"]):
            a = s["q"][first:first + nq, h].double() @ k[:, h // group].T / math.sqrt(d)
            if c["softcap"]:
                a = torch.tanh(a / c["softcap"]) * c["softcap"]
            a[hidden] = -math.inf
            heads.append(torch.softmax(a, 1) @ v[:, h // group])
        out.append(torch.stack(heads, 1))
        first += nq
    return torch.cat(out)


def _exact_norm(s, c):
    def rule(x, n):
        if c[n] == "none":
            return x
        if c[n] == "layer":
            var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
            return (x - mean) / torch.sqrt(var + EPS) * s[n + "_gamma"].double() + s[n + "_beta"].double()
        return x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["width"] + EPS) * s[n + "_gamma"].double()

    u = rule(s["y"].double(), "post")
    if c["gate_rows"] >= 0:
        row = torch.arange(c["rows"], device="cuda")
        u = u * s["gate"].double()[row // c["gate_rows"] if c["gate_rows"] else row * 0]
    r = s["x"].double() * c["residual_scale"] + u * c["block_scale"]
    return r, rule(r, "pre") if c["pre"] != "none" else None
