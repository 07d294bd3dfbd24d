"""GPU: attention_forward where scales and caps leave the usual range: a scale of
zero, which weighs all seen keys alike, and caps far above every score."""
import math

import pytest
import torch

from attention_reference import FN, ROUND, U32, assert_within, attention64, seen
from test_gpu_attention import _call, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("f32", 160), ("bf16", 64), ("bf16", 136)])
@pytest.mark.parametrize("q_len", [1, 12, 90])
@pytest.mark.parametrize("kw", [
    dict(causal=True), dict(kv_lens=[131, 40]), dict(window=30), dict(causal=True, softcap=20.0),
    dict(docs=[[0, 60, 150], [3, 100, 149]], causal=True),
], ids=lambda kw: "-".join(kw))
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-40])
def test_zero_scale_is_the_mean_of_the_seen_values(scale, kw, q_len, dtype, d):
    """Scores of zero, so the reference takes queries of zero; at 1e-40 scores are
    below 1e-37."""
    q, k, v = _inputs(2, q_len, 150, 4, 2, d, dtype, 3)
    lens = {n: kw[n] for n in ("kv_lens", "docs") if n in kw}
    c = {"dtype": dtype, **{n: x for n, x in kw.items() if n not in lens}}
    got = _call(q.cuda(), k.cuda(), v.cuda(), {**c, "scale": scale}, **lens)
    want, tol = attention64(torch.zeros_like(q), k, v, c, None, lens.get("kv_lens"), None, lens.get("docs"))
    assert_within(got, want, tol, f"{scale} {kw}")


def _capped64(q, k, v, cap, slopes, dtype):
    """Causal attention with capped scores and a bound on its error in which a
    score's cap costs 2^-21 of the score, whatever the cap."""
    b, q_len, hq, d = q.shape
    kv_len, group = k.shape[1], hq // k.shape[2]
    see = seen(q_len, kv_len, q_len, kv_len, causal=True, window=0, prefix=None, docs=None)
    dist = (kv_len - q_len + torch.arange(q_len)[:, None] - torch.arange(kv_len)[None, :]).abs().double()
    out = torch.zeros(q.shape, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for n in range(b):
        for h in range(hq):
            qq, kk, vv = q[n, :, h].double(), k[n, :, h // group].double(), v[n, :, h // group].double()
            s = cap * torch.tanh(qq @ kk.T * d ** -0.5 / cap)
            # The product's terms, the scale's and the cap's roundings, the function.
            err = (d + 8) * U32 * d ** -0.5 * (qq.abs() @ kk.abs().T) + FN * s.abs()
            if slopes is not None:
                bias = slopes[h].double() * dist
                s, err = s - bias, err + 4 * U32 * bias
            err = err + 4 * U32 * s.abs()
            w = torch.softmax(torch.where(see, s, -math.inf), 1)
            size = w @ vv.abs()
            e = torch.where(see & (w > 2.0 ** -20), err, 0.0).amax(1, keepdim=True)
            rel = 2 * e + 2 * FN + 2 * kv_len * U32 + (ROUND[dtype] if dtype == "bf16" else 0.0)
            out[n, :, h] = w @ vv
            tol[n, :, h] = size * rel + ROUND[dtype] * out[n, :, h].abs() + 2.0 ** -20 * kv_len * U32 + 1e-30
    return out, tol


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("q_len", [1, 12, 90])
@pytest.mark.parametrize("with_slopes", [False, True])
@pytest.mark.parametrize("cap", [600.0, 1e4, 1e6, 1e9, 1e30, 3e38])
def test_large_caps(cap, with_slopes, q_len, dtype, d):
    q, k, v = _inputs(2, q_len, 200, 4, 2, d, dtype, 7)
    slopes = torch.exp2(-2.0 * torch.arange(1, 5)).float() if with_slopes else None
    got = _call(q.cuda(), k.cuda(), v.cuda(), {"dtype": dtype, "causal": True, "softcap": cap}, slopes=slopes)
    want, tol = _capped64(q, k, v, cap, slopes, dtype)
    assert_within(got, want, tol, f"cap {cap}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("q_len", [1, 90])
@pytest.mark.parametrize("with_slopes", [False, True])
@pytest.mark.parametrize("cap", [1e-3, 1e-30, 1e-42])
def test_small_caps(cap, with_slopes, q_len, dtype):
    """Scores of at most the cap, also where the quotient scale / cap passes the
    largest fp32 number; one key's score is zero.  The bound lets the function
    be off by 2^-21 of the cap."""
    q, k, v = _inputs(1, q_len, 150, 4, 2, 64, dtype, 8)
    k[0, 3] = 0
    slopes = torch.exp2(-2.0 * torch.arange(1, 5)).float() if with_slopes else None
    c = {"dtype": dtype, "causal": True, "softcap": cap}
    got = _call(q.cuda(), k.cuda(), v.cuda(), c, slopes=slopes)
    want, tol = attention64(q, k, v, c, slopes=slopes)
    assert_within(got, want, tol, f"cap {cap}")


@pytest.mark.parametrize("kw", [dict(), dict(softcap=30.0, causal=True), dict(window=100, causal=True)],
                         ids=lambda kw: "-".join(kw) or "plain")
@pytest.mark.parametrize("b,q_len,kv_len,hq,hk,d", [(3, 1, 700, 8, 2, 128), (2, 4, 300, 4, 2, 64), (1, 2, 5000, 16, 2, 256),
                                                    (4, 1, 33, 6, 6, 96)])
def test_few_rows_keep_16_bits_of_the_weights(b, q_len, kv_len, hq, hk, d, kw):
    """bf16: the bound of fp32 weights, 2^-16 of the values' weighted size for the
    weights' two parts (each off by 2^-8 of what it stands for), and the output's
    rounding."""
    q, k, v = _inputs(b, q_len, kv_len, hq, hk, d, "bf16", 9)
    got = _call(q.cuda(), k.cuda(), v.cuda(), {"dtype": "bf16", **kw})
    want, tol = attention64(q, k, v, {"dtype": "f32", **kw})
    size, _ = attention64(q, k, v.abs(), {"dtype": "f32", **kw})
    assert_within(got, want, tol + 2.0 ** -16 * size + ROUND["bf16"] * want.abs())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("b,q_len,kv_len,hq,hk,d", [(3, 1, 700, 8, 2, 128), (2, 4, 300, 4, 2, 64), (1, 2, 900, 16, 2, 256),
                                                    (4, 1, 33, 6, 6, 96), (1, 70, 200, 4, 2, 64)])
@pytest.mark.parametrize("causal", [False, True])
def test_infinities_that_all_rows_see(causal, b, q_len, kv_len, hq, hk, d, dtype):
    """Also where weights have few bits or are powers of two: an infinity stays
    one, and its sign; both signs, or NaN, make NaN."""
    q, k, v = _inputs(b, q_len, kv_len, hq, hk, d, dtype, 10)
    q[0, 0] = 0                       # equal scores: weights of one
    last = kv_len - q_len             # seen by all rows, causal or not
    v[0, last // 2, 0, 1] = math.inf
    v[:, last, hk - 1, 2] = -math.inf
    v[0, 0, 0, 3], v[0, last // 3, 0, 3] = math.inf, -math.inf
    v[0, 1 % (last + 1), hk - 1, d - 1] = math.nan
    c = {"dtype": dtype, "causal": causal}
    got = _call(q.cuda(), k.cuda(), v.cuda(), c)
    want, tol = attention64(q, k, v, c)
    assert torch.isinf(want).any() and torch.isnan(want).any()
    assert_within(got, want, tol)
