"""GPU: paged_attention_forward of single tokens of many sequences of which a few are long."""
import pytest
import torch

from attention_reference import TYPES, assert_within
from decoder_reference import paged64, random_cache

pytestmark = pytest.mark.gpu

KINDS = [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32"), ("f32", "e4m3")]


def _run(lens, long_at, hq, hk, d, dtype, cache, check, q_lens=None):
    """Sequences share pages in an order of their own; those of `check` are held against the definition."""
    import convolution_conv2d_forward_amd as m
    ps, n_pages, batch = 16, 80, len(lens)
    lens = list(lens)
    for b, n in long_at.items():
        lens[b] = n
    q_lens = q_lens or [1] * batch
    offsets = [sum(q_lens[:b]) for b in range(batch + 1)]
    got, values = random_cache(n_pages, ps, hk, d, dtype, cache, 3)
    g = torch.Generator().manual_seed(batch)
    table = torch.randint(0, n_pages, (batch, -(-max(lens) // ps)), generator=g, dtype=torch.int32)
    q = (2 * torch.randn(offsets[-1], hq, d, generator=g)).to(TYPES[dtype])
    desc = m.paged_attention_desc_create(m.make_paged_attention_params(hq, hk, d, ps, dtype=dtype, cache_dtype=cache))
    n = m.paged_attention_workspace_bytes(desc, offsets[-1], batch, table.shape[1])
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    dev = [None if got[x] is None else got[x].cuda() for x in ("k", "v", "ks", "vs")]
    m.paged_attention_forward(desc, q.cuda(), ints(offsets), ints(lens), table.cuda(), *dev, out,
                              workspace=torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None)
    assert (out != 9).all()
    for b in check:
        rows = slice(offsets[b], offsets[b + 1])
        want, tol, _ = paged64(q[rows], [0, q_lens[b]], [lens[b]], table[b:b + 1], values, dict(dtype=dtype))
        assert_within(out[rows], want, tol, f"sequence {b} of {lens[b]} keys")


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("batch,hq,hk,d", [(256, 16, 8, 64), (300, 32, 32, 32), (1000, 8, 8, 128), (1024, 2, 1, 64)])
def test_a_long_sequence_among_many(batch, hq, hk, d, dtype, cache):
    lens = [1 + 37 * b % 130 for b in range(batch)]
    _run(lens, {0: 5000, batch // 2: 3001, batch - 1: 999}, hq, hk, d, dtype, cache,
         [0, 1, 2, 63, 64, batch // 2 - 1, batch // 2, batch // 2 + 1, batch - 2, batch - 1])


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_more_heads_than_records_are_left_for(dtype, cache):
    """1000 sequences of 64 heads: taken whole."""
    _run([1 + b % 40 for b in range(1000)], {0: 700}, 64, 64, 32, dtype, cache, [0, 1, 500, 998, 999])


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_a_few_tokens_each_and_none(dtype, cache):
    """Up to four tokens, sequences without new ones or without keys among them."""
    q_lens = [(0, 1, 4, 2)[b % 4] for b in range(400)]
    _run([41 * b % 200 for b in range(400)], {1: 4000, 2: 2500}, 8, 8, 64, dtype, cache, [1, 2, 3, 5, 6, 399], q_lens)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_captured_while_lengths_change(cache):
    """One captured call of 300 sequences: none is long, the first and last are, another is; other work between."""
    import convolution_conv2d_forward_amd as m
    ps, n_pages, batch, hq, hk, d = 16, 80, 300, 16, 8, 64
    got, values = random_cache(n_pages, ps, hk, d, "bf16", cache, 3)
    g = torch.Generator().manual_seed(1)
    table = torch.randint(0, n_pages, (batch, 250), generator=g, dtype=torch.int32)
    dev = [None if got[x] is None else got[x].cuda() for x in ("k", "v", "ks", "vs")]
    q, out = torch.zeros(batch, hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(batch, hq, d, dtype=torch.bfloat16, device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    off, lens, tab = ints(list(range(batch + 1))), ints([1] * batch), table.cuda()
    desc = m.paged_attention_desc_create(m.make_paged_attention_params(hq, hk, d, ps, dtype="bf16", cache_dtype=cache))
    ws = torch.zeros(m.paged_attention_workspace_bytes(desc, batch, batch, 250), dtype=torch.uint8, device="cuda")
    call = lambda: m.paged_attention_forward(desc, q, off, lens, tab, *dev, out, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for long_at in ({}, {0: 4000, 299: 2500}, {150: 3999}, {}):
        now = [1 + 7 * b % 60 for b in range(batch)]
        for b, n in long_at.items():
            now[b] = n
        x = torch.randn(batch, hq, d, generator=g).to(torch.bfloat16)
        q.copy_(x)
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        out.fill_(float("nan"))
        graph.replay()
        for b in (0, 1, 150, 298, 299):
            want, tol, _ = paged64(x[b:b + 1], [0, 1], now[b:b + 1], table[b:b + 1], values, dict(dtype="bf16"))
            assert_within(out[b:b + 1], want, tol, f"sequence {b} of {now[b]} keys")
        assert torch.isfinite(out).all()
        torch.cuda.synchronize()
