"""GPU: calls of more workgroups than one launch holds (2^32 work-items): short
sequences, tokens and rows by the million, each checked whole."""
import pytest
import torch

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


def cc():
    import convolution_conv2d_forward_amd as m
    return m


def test_attention_over_millions_of_short_sequences():
    """2^19 + 3 sequences of one token and 32 key heads: the only key's weight is
    one, so a row is its value, or zero where lengths or documents leave no key."""
    m, b, h, d = cc(), (1 << 19) + 3, 32, 8
    q = torch.zeros((b, 1, h, d), dtype=bf16, device="cuda")
    k, v = (torch.randn((b, 1, h, d), device="cuda").to(bf16) for _ in "kv")
    lens = (torch.arange(b, device="cuda") % 7 != 3).to(torch.int32)
    docs = torch.zeros((b, 2), dtype=torch.int32, device="cuda")
    docs[:, 1] = (torch.arange(b, device="cuda") % 5 != 1).to(torch.int32)
    desc = m.attention_desc_create(m.make_attention_params(
        h, h, d, q_strides=q.stride()[:3], k_strides=k.stride()[:3], v_strides=v.stride()[:3],
        out_strides=q.stride()[:3], dtype="bf16"))
    assert m.attention_workspace_bytes(desc, b, 1, 1) == 0
    out = torch.full_like(q, float("nan"))
    m.attention_forward(desc, q, k, v, out, kv_lens=lens, doc_offsets=docs)
    assert torch.equal(out, v * (lens * docs[:, 1]).to(bf16)[:, None, None, None])


@pytest.mark.parametrize("d,tokens", [(2, 22_400_000), (8, (1 << 26) + 77)])
@pytest.mark.parametrize("with_slots", [False, True])
def test_rope_over_millions_of_tokens(with_slots, d, tokens):
    """One query, key and value head, of 2 elements (a wave each) or 8 (a wave a
    token); positions 0 and 1 by turns."""
    m = cc()
    qkv = torch.randn((tokens, 3 * d), device="cuda").to(bf16)
    pos = (torch.arange(tokens, device="cuda") % 3 == 1).to(torch.int32)
    slots = (tokens - 1 - torch.arange(tokens, device="cuda")).to(torch.int32) if with_slots else None
    q, k, v = (torch.full((tokens, 1, d), float("nan"), dtype=bf16, device="cuda") for _ in "qkv")
    desc = m.qk_rope_desc_create(m.make_qk_rope_params(1, 1, d, rotary_dim=2, dtype="bf16"))
    m.qk_rope_forward(desc, qkv, None, None, pos, slots, q, k, v)
    if with_slots:
        k, v = k.flip(0), v.flip(0)
    assert torch.equal(v[:, 0], qkv[:, 2 * d:])
    for got, x in ((q, qkv[:, :d]), (k, qkv[:, d:2 * d])):
        got = got[:, 0]
        assert torch.equal(got[:, 2:], x[:, 2:])
        still = pos == 0
        assert torch.equal(got[still, :2], x[still, :2])
        a, b = x[~still, 0].double(), x[~still, 1].double()
        one = torch.ones((), dtype=torch.float64, device="cuda")
        for have, want in ((got[~still, 0], a * one.cos() - b * one.sin()), (got[~still, 1], b * one.cos() + a * one.sin())):
            # One rounding to bf16, and the products' and functions' errors.
            assert ((have.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * (a.abs() + b.abs())).all()


@pytest.mark.parametrize("shift", [0, 1])
def test_linear_over_a_billion_rows(shift):
    """Rows of one element, at 2-byte boundaries, so through registers: a
    workgroup for each 64."""
    m, rows = cc(), (1 << 30) + 1000
    x = torch.empty(rows + shift, dtype=bf16, device="cuda")
    x.view(torch.int16).random_(128, 20000)   # normal numbers of all sizes
    x = x[shift:, None]
    y = torch.full((rows, 1), float("nan"), dtype=bf16, device="cuda")
    desc = m.linear_desc_create(m.make_linear_params(1, 1, dtype="bf16"))
    m.linear_forward(desc, x, torch.ones((1, 1), dtype=bf16, device="cuda"), None, None, y)
    assert torch.equal(x, y)
