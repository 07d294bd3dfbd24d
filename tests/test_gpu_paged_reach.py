"""GPU: paged_attention_forward over 2^30 keys, as many as a call takes, whose stretches can be told apart: a stretch that
is left out or taken twice shows in every element."""
import pytest
import torch

from attention_reference import TYPES
from decoder_reference import E4M3, quantise64

pytestmark = pytest.mark.gpu

PS, PAGES = 4096, (1 << 30) // 4096
# (first page, share of the output): single pages at the beginning, at 2^29 keys and at the end, whose values are so
# large that each is a share of 0.3, and quarters of the keys with shares of 0.1 in all.
STRETCHES = [(0, 0.3), (1, 0.01), (PAGES // 4, 0.02), (PAGES // 2, 0.3), (PAGES // 2 + 1, 0.03), (3 * PAGES // 4, 0.04),
             (PAGES - 1, 0.3)]


def _parts(k, v, q, counts, scale):
    """Per row: sums of weights and of weighted values [stretch][row], the last page's as its rows see it."""
    rows, last = q.shape[0], len(counts) - 1
    total, out = [], []
    for s, n in enumerate(counts):
        w = torch.exp(scale * q @ k[s].T)
        if s == last:   # row i is rows - 1 - i keys before the end
            w = torch.where(torch.arange(PS)[None] < PS - rows + 1 + torch.arange(rows)[:, None], w, 0.0)
        total.append(n * w.sum(1))
        out.append(n * w @ v[s])
    return torch.stack(total), torch.stack(out)


@pytest.mark.parametrize("cache,d", [("bf16", 8), ("e4m3", 16)])
@pytest.mark.parametrize("q_len,tol", [(1, 2.0 ** -6), (20, 2.0 ** -4)])
def test_every_stretch_of_the_longest_sequence(q_len, tol, cache, d):
    """A lane adds up to 2^17 weights (single tokens) or 2^18.5 (chunks) in fp32, and as many products: each addition is
    off by 2^-24 of the sum, twice; values are positive, so a sum is never above its end.  The weights' and the output's
    own rounding to bf16 come to it."""
    g = torch.Generator().manual_seed(d + q_len)
    ends = [p for p, _ in STRETCHES[1:]] + [PAGES]
    counts = [end - p for (p, _), end in zip(STRETCHES, ends)]
    k = torch.randn(len(counts), PS, 1, d, generator=g)
    v = 1 + 0.25 * torch.rand(len(counts), PS, 1, d, generator=g)
    v *= torch.tensor([share * PAGES / n for (_, share), n in zip(STRETCHES, counts)])[:, None, None, None]
    pages, scales, values = [], [None, None], []
    for x in (k.to(torch.bfloat16), v.to(torch.bfloat16)):
        if cache == "e4m3":
            codes, e = quantise64(x)
            pages.append(codes.float().to(E4M3).cuda())
            scales[len(pages) - 1] = (e + 127).to(torch.uint8).cuda()
            values.append(torch.ldexp(codes, e[..., None])[:, :, 0])
        else:
            pages.append(x.cuda())
            values.append(x.double()[:, :, 0])
    q = torch.randn(q_len, 1, d, generator=g).to(torch.bfloat16)
    total, out = _parts(*values, q[:, 0].double(), counts, d ** -0.5)
    want = out.sum(0) / total.sum(0)[:, None]
    bound = (tol + 2.0 ** -7) * want
    for s in range(len(counts)):   # left out, or twice
        for f in (-1, 1):
            other = (out.sum(0) + f * out[s]) / (total.sum(0) + f * total[s])[:, None]
            assert ((other - want).abs() > 1.5 * bound).all(), (s, f)
    table = torch.repeat_interleave(torch.arange(len(counts), dtype=torch.int32), torch.tensor(counts))[None].cuda()
    import convolution_conv2d_forward_amd as m
    desc = m.paged_attention_desc_create(m.make_paged_attention_params(1, 1, d, PS, dtype="bf16", cache_dtype=cache))
    n = m.paged_attention_workspace_bytes(desc, q_len, 1, PAGES)
    got = torch.full((q_len, 1, d), 9e9, dtype=TYPES["bf16"], device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    m.paged_attention_forward(desc, q.cuda(), ints([0, q_len]), ints([1 << 30]), table, *pages, *scales, got,
                              workspace=torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None)
    off = (got[:, 0].double().cpu() - want).abs() / bound
    assert (off <= 1).all(), float(off.max())
