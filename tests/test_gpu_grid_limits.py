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
