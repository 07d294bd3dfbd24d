"""Plain 64-bit definitions of linear, qk_rope and attention, on the CPU, and
the error bounds their tests use.

Bounds are derived from the number formats: a rounding to bf16 is off by at
most 2^-8 relative, one to fp32 by 2^-24; an fp32 sum of n terms by n * 2^-24
of the terms' absolute sum; library and hardware functions of one argument by
2^-21 of their scale."""
import math

import torch

U32, FN = 2.0 ** -24, 2.0 ** -21
ROUND = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def act64(name, v, alpha=0.01, clip=(-math.inf, math.inf)):
    if name == "none":
        return v
    if name == "relu":
        return v.clamp(min=0)
    if name == "leaky_relu":
        return torch.where(v >= 0, v, alpha * v)
    if name == "clip":
        return v.clamp(*clip)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    raise ValueError(name)


def linear64(x, w, bias, residual, dtype, act="none", alpha=0.01, clip=(-math.inf, math.inf)):
    """(y, bound on |error|) for CPU tensors of the call's types."""
    x, w = x.double(), w.double()
    v, size = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        v, size = v + bias.double(), size + bias.double().abs()
    y = act64(act, v, alpha, clip)
    # |act'| <= 1.13 for every activation here; the functions' own error goes
    # with the argument's size.
    tol = 1.13 * (x.shape[1] + 2) * U32 * size + FN * v.abs() * (act in ("silu", "gelu", "gelu_tanh")) + 2 * U32 * y.abs()
    if residual is not None:
        y = y + residual.double()
    return y, tol + ROUND[dtype] * y.abs() + 2 * U32 * y.abs() + 1e-30


def rope_frequencies(c):
    r, out = c["rotary_dim"], []
    factor = 1.0
    for i in range(r // 2):
        f = c["theta"] ** (-2.0 * i / r)
        if c["scaling"] == "linear":
            f /= c["factor"]
        elif c["scaling"] == "yarn":
            t = lambda n: r * math.log(c["original_len"] / (2 * math.pi * n)) / (2 * math.log(c["theta"]))  # noqa: E731
            lo, hi = max(math.floor(t(32.0)), 0), min(math.ceil(t(1.0)), r - 1)
            ramp = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = f * (1 - ramp) + f / c["factor"] * ramp
            factor = 0.1 * math.log(c["factor"]) + 1
        out.append(f)
    return torch.tensor(out, dtype=torch.float64), factor


def rope64(x, gamma, positions, c):
    """(rotated, bound) of x [tokens, heads, head_dim] (CPU, the call's type)."""
    d, r = x.shape[-1], c["rotary_dim"]
    x = x.double()
    if gamma is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + c["eps"]) * gamma.double()
    f, factor = rope_frequencies(c)
    ang = positions.double()[:, None, None] * f
    cos, sin = torch.cos(ang) * factor, torch.sin(ang) * factor
    y, size = x.clone(), x.abs()
    if c["layout"] == "half":
        i0, i1 = slice(0, r // 2), slice(r // 2, r)
    else:
        i0, i1 = slice(0, r, 2), slice(1, r, 2)
    a, b = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = a * cos - b * sin, b * cos + a * sin
    both = (a.abs() + b.abs()) * factor
    size[..., i0], size[..., i1] = both, both
    norm = (d + 8) * U32 if gamma is not None else 0.0
    return y, size * (norm + 2 * FN) + ROUND[c["dtype"]] * y.abs() + 1e-30


def seen(q_len, kv_len, nq, nk, *, causal, window, prefix, docs):
    """Boolean [q_len, kv_len]: the header's conditions, one by one."""
    i = torch.arange(q_len)[:, None]
    j = torch.arange(kv_len)[None, :]
    p = nk - nq + i
    see = (i < nq) & (j < nk)
    if causal:
        order = j <= p
        if prefix is not None:
            order = order | (j < prefix)
        see = see & order
    if window:
        see = see & ((p - j).abs() < window)
    if docs is not None:
        same = torch.zeros_like(see)
        for lo, hi in zip(docs, docs[1:]):
            same |= (p >= lo) & (p < hi) & (j >= lo) & (j < hi)
        see = see & same
    return see


def attention64(q, k, v, c, q_lens=None, kv_lens=None, prefix=None, docs=None, slopes=None):
    """(out, bound) of q [b, q_len, hq, d], k and v [b, kv_len, hk, d] (CPU).
    Elements that a row does not see are left out, not multiplied by 0."""
    b, q_len, hq, d = q.shape
    kv_len, hk = k.shape[1], k.shape[2]
    scale = c.get("scale") or d ** -0.5
    cap, u = c.get("softcap", 0.0), ROUND[c["dtype"]]
    out = torch.zeros((b, q_len, hq, d), dtype=torch.float64)
    tol = torch.zeros_like(out)
    for n in range(b):
        nq = q_len if q_lens is None else min(max(q_lens[n], 0), q_len)
        nk = kv_len if kv_lens is None else min(max(kv_lens[n], 0), kv_len)
        see = seen(q_len, kv_len, nq, nk, causal=c.get("causal", False), window=c.get("window", 0),
                   prefix=None if prefix is None else prefix[n], docs=None if docs is None else docs[n])
        p = nk - nq + torch.arange(q_len)[:, None]
        dist = (p - torch.arange(kv_len)[None, :]).abs().double()
        used = see.any(0)
        for h in range(hq):
            kk = torch.where(used[:, None], k[n, :, h // (hq // hk)].double(), 0.0)
            vv = torch.where(used[:, None], v[n, :, h // (hq // hk)].double(), 0.0)
            qq = q[n, :, h].double()
            s = scale * qq @ kk.T
            err = (d + 8) * U32 * abs(scale) * (qq.abs() @ kk.abs().T)
            if cap:
                s = cap * torch.tanh(s / cap)
                err = err + cap * FN
            if slopes is not None:
                s = s - slopes[h].double() * dist
                err = err + 4 * U32 * slopes[h].double().abs() * dist
            err = err + 4 * U32 * s.abs()
            s = torch.where(see, s, -math.inf)
            top = s.amax(1, keepdim=True)
            w = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
            total = w.sum(1, keepdim=True)
            w = w / torch.where(total == 0, 1.0, total)
            # Non-finite values reach exactly the rows that see them.
            bad = ~torch.isfinite(vv)
            if bad.any():
                o = torch.stack([torch.where(see[i][:, None], w[i][:, None] * vv, 0.0).sum(0) for i in range(q_len)])
            else:
                o = w @ vv
            size = w @ torch.where(bad, 0.0, vv.abs())
            # A weight is off by its score's error (which counts twice: also in
            # the sum), the exponential's, the sum's, and for bf16 by its own
            # rounding before the product.  Weights below 2^-20 add nothing
            # of a score's error that is seen, so far keys' larger errors do
            # not count.
            e = torch.where(see & (w > 2.0 ** -20), err, 0.0).amax(1, keepdim=True)
            rel = 2 * e + 2 * FN + 2 * kv_len * U32 + (u if c["dtype"] == "bf16" else 0.0)
            out[n, :, h] = o
            tol[n, :, h] = size * rel + u * o.abs() + 2.0 ** -20 * kv_len * U32 + 1e-30
    return out, tol


def assert_within(got, want, tol, what=""):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (got.shape, want.shape)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    fine = ~(nan | inf)
    assert torch.isfinite(got[fine]).all(), f"{what}: non-finite output"
    if fine.any():
        over = ((got - want).abs() - tol)[fine]
        at = int(over.argmax())
        assert over[at] <= 0, (f"{what}: off by {float((got - want).abs()[fine][at]):.3e} where "
                               f"{float(tol[fine][at]):.3e} is allowed (value {float(want[fine][at]):.4g}); "
                               f"{int((over > 0).sum())} of {over.numel()} beyond")
