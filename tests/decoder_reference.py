"""Plain 64-bit definitions of the paged cache, of attention over it and of block_norm, on the CPU, and the error bounds
their tests use (the same reasoning as attention_reference's)."""
import math

import torch

from attention_reference import FN, ROUND, TYPES, U32

E4M3 = torch.float8_e4m3fn


# -------------------------------------------------------------- the cache --

def quantise64(x):
    """(values of the codes, exponents) of rows x [..., d]: see kv_cache_store."""
    x = x.double()
    fine = torch.isfinite(x)
    top = torch.where(fine, x.abs(), 0.0).amax(-1)
    e = torch.full(top.shape, -117, dtype=torch.int64)
    for i, t in enumerate(top.flatten().tolist()):
        if t > 0:
            m, n = math.frexp(t)   # t = m 2^n
            e.view(-1)[i] = min(max(n - 9 if m <= 0.875 else n - 8, -117), 119)
    v = torch.ldexp(torch.where(fine, x, 0.0), -e[..., None]).clamp(-448, 448)
    # Steps of 2^-3 of the power of two below the value, 2^-9 at least.
    _, n = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (n - 1).clamp(min=-6) - 3)
    return torch.where(fine, torch.round(v / step) * step, math.nan), e


def random_cache(n_pages, page_size, heads, d, dtype, cache, seed=0, scale=1.0):
    """Pages of random keys and values: {"k": pages, "v": ..., "ks": scales or None, "vs": ...} on the CPU, and their
    values in 64 bits, {"k": ..., "v": ...}."""
    g = torch.Generator().manual_seed(seed)
    got, values = {}, {}
    for n in "kv":
        x = (scale * torch.randn(n_pages, page_size, heads, d, generator=g)).to(TYPES[dtype])
        got[n + "s"] = None
        if cache == "e4m3":
            codes, e = quantise64(x)
            got[n], got[n + "s"] = codes.float().to(E4M3), (e + 127).to(torch.uint8)
            values[n] = torch.ldexp(codes, e[..., None])
        else:
            got[n], values[n] = x, x.double()
    return got, values


def tables(lens, page_size, n_pages, max_pages, seed=0):
    """A page table for sequences of these lengths: pages in random order, -1 behind a sequence's own."""
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    t, at = torch.full((len(lens), max_pages), -1, dtype=torch.int32), 0
    for b, n in enumerate(lens):
        need = -(-max(n, 0) // page_size)
        t[b, :need] = torch.tensor(order[at:at + need], dtype=torch.int32)
        at += need
    assert at <= n_pages
    return t


def sequence64(values, table, length, page_size):
    """(rows [length, heads, d], which of them there are) of one sequence."""
    page = table.long()[torch.arange(length) // values.shape[1]]
    there = (page >= 0) & (page < values.shape[0])
    if not there.any():
        return torch.zeros((length,) + tuple(values.shape[2:]), dtype=torch.float64), there
    rows = values[page.clamp(0, values.shape[0] - 1), torch.arange(length) % values.shape[1]]
    return torch.where(there[:, None, None], rows, 0.0), there


# -------------------------------------------------------------- attention --

def seen64(nq, nk, window, sinks):
    """Boolean [nq, nk]: the header's conditions, one by one."""
    p, j = nk - nq + torch.arange(nq)[:, None], torch.arange(nk)[None, :]
    see = j <= p
    if window:
        see = see & ((p - j < window) | (j < sinks))
    return see


def paged64(q, offsets, lens, table, values, c):
    """(out, bound, rows that belong to a sequence) of q [tokens, heads_q, d] (CPU).  Elements that a row does not see
    are left out, not multiplied by 0."""
    tokens, hq, d = q.shape
    k_all, v_all = values["k"], values["v"]
    ps, hk = k_all.shape[1], k_all.shape[2]
    scale, cap, u = c.get("scale"), c.get("softcap", 0.0), ROUND[c["dtype"]]
    scale = d ** -0.5 if scale is None else scale
    out, tol = torch.zeros((tokens, hq, d), dtype=torch.float64), torch.zeros((tokens, hq, d), dtype=torch.float64)
    mine = torch.zeros(tokens, dtype=torch.bool)
    clamp = lambda x: min(max(x, 0), tokens)  # noqa: E731
    for b, n in enumerate(lens):
        first, nq = clamp(offsets[b]), clamp(offsets[b + 1]) - clamp(offsets[b])
        if nq <= 0:
            continue
        nk = min(max(n, 0), table.shape[1] * ps)
        (k, there), (v, _) = sequence64(k_all, table[b], nk, ps), sequence64(v_all, table[b], nk, ps)
        see = seen64(nq, nk, c.get("window", 0), c.get("sinks", 0)) & there
        used = see.any(0)
        k, v = torch.where(used[:, None, None], k, 0.0), torch.where(used[:, None, None], v, 0.0)
        mine[first:first + nq] = True
        for h in range(hq):
            kk, vv, qq = k[:, h // (hq // hk)], v[:, h // (hq // hk)], q[first:first + nq, h].double()
            s = scale * qq @ kk.T
            err = (d + 8) * U32 * abs(scale) * (qq.abs() @ kk.abs().T)
            if cap:
                s = cap * torch.tanh(s / cap)
                err = err + cap * FN
            err = err + 4 * U32 * s.abs()
            s = torch.where(see, s, -math.inf)
            top = s.amax(1, keepdim=True) if nk else torch.full((nq, 1), -math.inf, dtype=torch.float64)
            w = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
            total = w.sum(1, keepdim=True)
            w = w / torch.where(total == 0, 1.0, total)
            bad = ~torch.isfinite(vv)
            if bad.any():
                o = torch.stack([torch.where(see[i][:, None], w[i][:, None] * vv, 0.0).sum(0) for i in range(nq)])
            else:
                o = w @ vv
            size = w @ torch.where(bad, 0.0, vv.abs())
            # A weight is off by its score's error (which counts twice: also in the sum), the exponential's, the sum's,
            # and for bf16 by its own rounding before the product.
            e = torch.where(see & (w > 2.0 ** -20), err, 0.0).amax(1, keepdim=True) if nk else 0.0
            rel = 2 * e + 2 * FN + 2 * nk * U32 + (u if c["dtype"] == "bf16" else 0.0)
            out[first:first + nq, h] = o
            tol[first:first + nq, h] = size * rel + u * o.abs() + 2.0 ** -20 * nk * U32 + 1e-30
    return out, tol, mine


# ------------------------------------------------------------- block norm --

def _norm64(x, err, kind, gamma, beta, eps):
    """The norm of x and what errors of up to `err` in it and fp32's own make of it."""
    n = x.shape[-1]
    if kind == "none":
        return x, err
    if kind == "layer":
        mean = x.mean(-1, keepdim=True)
        err = err + err.mean(-1, keepdim=True) + n * U32 * x.abs().mean(-1, keepdim=True)
        x = x - mean
        err = err + U32 * x.abs()
    ms = (x * x).mean(-1, keepdim=True)
    off = (2 * x.abs() * err + err * err).mean(-1, keepdim=True) + (n + 2) * U32 * ms
    r = 1 / torch.sqrt(ms + eps)
    rel = 0.5 * off / (ms + eps) + 4 * U32
    g = gamma.double()
    y = x * r * g
    err = (err + x.abs() * rel) * r * g.abs() + 4 * U32 * y.abs()
    if beta is not None:
        y = y + beta.double()
        err = err + U32 * y.abs()
    return y, err


def block_norm64(y, x, gate, v, c):
    """((residual, bound), (out, bound) or None) for CPU tensors; v: post_gamma, post_beta, pre_gamma, pre_beta."""
    rows, u = y.shape[0], ROUND[c["dtype"]]
    a, err = _norm64(y.double(), torch.zeros(y.shape, dtype=torch.float64), c["post"], v[0], v[1], c["eps"])
    if gate is not None:
        g = gate.double()
        g = g[torch.arange(rows) // c["gate_rows"]] if c["gate_rows"] else g
        a, err = a * g, err * g.abs()
        err = err + U32 * a.abs()
    xs, bs = c["residual_scale"], c["block_scale"]
    r = xs * x.double() + bs * a
    err = err * abs(bs) + 3 * U32 * ((xs * x.double()).abs() + (bs * a).abs())
    tol = err + u * (r.abs() + err) + 1e-30
    if c["pre"] == "none":
        return (r, tol), None
    o, err = _norm64(r, err, c["pre"], v[2], v[3], c["eps"])
    return (r, tol), (o, err + u * (o.abs() + err) + 1e-30)
