"""GPU: attention_forward over keys 2^24 elements and more apart, which many rows
walk with the kernel for any strides: every width, mask and bias, and values that
no row sees.  k and v lie side by side in one buffer, of which only their own
elements are written."""
import pytest
import torch

from attention_reference import TYPES, assert_within, attention64
from test_gpu_attention import _call, _inputs

pytestmark = pytest.mark.gpu
STRIDE = 1 << 24


def _far(k, v):
    """k and v on the GPU, STRIDE elements from a token to the next, the heads
    and sequences of a token after each other."""
    b, n, h, d = k.shape
    buf = torch.empty((n - 1) * STRIDE + 2 * b * h * d, dtype=k.dtype, device="cuda")
    out = []
    for i, x in enumerate((k, v)):
        t = buf.as_strided((b, n, h, d), (h * d, STRIDE, d, 1), i * b * h * d)
        t.copy_(x)
        out.append(t)
    return out


def _check(q, k, v, c, **lens):
    got = _call(q.cuda(), *_far(k, v), c, **lens)
    want, tol = attention64(q, k, v, c, lens.get("q_lens"), lens.get("kv_lens"), lens.get("prefix"), lens.get("docs"),
                            lens.get("slopes"))
    assert_within(got, want, tol, f"{c} {lens}")


DIMS = {"f32": [4, 32, 48, 80, 100, 128, 200, 256], "bf16": [8, 32, 40, 80, 96, 128, 192, 256]}


@pytest.mark.parametrize("dtype,d", [(t, d) for t, ds in DIMS.items() for d in ds])
@pytest.mark.parametrize("softcap", [0.0, 30.0, 1e4])
def test_head_dims(softcap, dtype, d):
    _check(*_inputs(1, 45, 70, 4, 2, d, dtype, 2), {"dtype": dtype, "causal": True, "softcap": softcap})


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("f32", 128), ("bf16", 64), ("bf16", 96)])
@pytest.mark.parametrize("kw", [
    dict(), dict(slopes=True, softcap=20.0), dict(window=30), dict(window=7, causal=True), dict(prefix=[40, 0], causal=True),
    dict(docs=[[0, 20, 20, 50, 66], [3, 10, 40, 60, 66]], causal=True, slopes=True), dict(scale=0.0, causal=True),
    dict(q_lens=[50, 7], kv_lens=[66, 0], causal=True), dict(q_lens=[9, 50], kv_lens=[33, 20]),
], ids=lambda kw: "-".join(kw) or "plain")
def test_masks_and_biases(kw, dtype, d):
    kw = dict(kw)
    lens = {n: kw.pop(n) for n in ("q_lens", "kv_lens", "prefix", "docs") if n in kw}
    if kw.pop("slopes", False):
        lens["slopes"] = torch.exp2(-2.0 * torch.arange(1, 5)).float()
    q, k, v = _inputs(2, 50, 66, 4, 2, d, dtype, 3)
    if kw.get("scale") == 0.0:   # for the reference: scores of zero
        q = torch.zeros_like(q)
        got = _call(_inputs(2, 50, 66, 4, 2, d, dtype, 3)[0].cuda(), *_far(k, v), {"dtype": dtype, **kw})
        want, tol = attention64(q, k, v, {"dtype": dtype, "causal": True})
        assert_within(got, want, tol)
        return
    _check(q, k, v, {"dtype": dtype, **kw}, **lens)


@pytest.mark.parametrize("dtype,d", [("f32", 48), ("f32", 160), ("bf16", 64), ("bf16", 136)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_unseen_garbage_does_not_spread(bad, dtype, d):
    c = {"dtype": dtype, "causal": True, "window": 25}
    q, k, v = _inputs(2, 60, 70, 4, 2, d, dtype, 4)
    docs, lens = [[0, 30, 70]] * 2, [70, 51]
    k[1, 51:] = bad
    v[1, 51:] = bad
    v[0, 69, 0, 3] = bad       # seen by the last row alone
    v[0, 35, 1, d - 1] = bad
    k[0, 12] = bad if bad != bad else 0.0
    _check(q, k, v, c, kv_lens=lens, docs=docs)
