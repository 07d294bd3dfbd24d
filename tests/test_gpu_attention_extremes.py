"""GPU: attention_forward where scales leave the usual range: a scale of zero
weighs all seen keys alike."""
import pytest
import torch

from attention_reference import assert_within, attention64
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
