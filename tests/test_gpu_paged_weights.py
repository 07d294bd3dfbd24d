"""GPU: the softmax weights of paged_attention_forward in bf16: 16 bits of them meet the values in sequences of up to 16
rows of a key head, whatever else the batch holds."""
import math

import pytest
import torch

from decoder_reference import E4M3, sequence64, tables

pytestmark = pytest.mark.gpu

U, U32, FN = 2.0 ** -8, 2.0 ** -24, 2.0 ** -21
BF16 = torch.bfloat16


def cc():
    import convolution_conv2d_forward_amd as m
    return m


def _ints(v):
    return torch.as_tensor(v, dtype=torch.int32).cuda()


def _run(q, q_lens, lens, table, pages, scales, hk, cache, **c):
    m = cc()
    tokens, hq, d = q.shape
    desc = m.paged_attention_desc_create(m.make_paged_attention_params(hq, hk, d, pages[0].shape[1], dtype="bf16",
                                                                       cache_dtype=cache, **c))
    n = m.paged_attention_workspace_bytes(desc, tokens, len(lens), table.shape[1])
    out = torch.full_like(q, 9.0, device="cuda")
    offsets = [sum(q_lens[:i]) for i in range(len(q_lens) + 1)]
    m.paged_attention_forward(desc, q.cuda(), _ints(offsets), _ints(lens), _ints(table), *pages, *scales, out,
                              workspace=torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None)
    return out.cpu().double()


def _cache(n_pages, ps, hk, d, cache, seed):
    """Values and keys that both cache types hold exactly (4 bits, scales of one), and their 64-bit values."""
    g = torch.Generator().manual_seed(seed)
    got = {n: torch.randn(n_pages, ps, hk, d, generator=g).to(E4M3) for n in "kv"}
    values = {n: got[n].double() for n in "kv"}
    if cache == "e4m3":
        one = torch.full((n_pages, ps, hk), 127, dtype=torch.uint8).cuda()
        return [got["k"].cuda(), got["v"].cuda()], [one, one], values
    return [got[n].float().to(BF16).cuda() for n in "kv"], [None, None], values


# Rows of a key head (4 query heads share one): 4, 8, 12, 16 in short sequences; the others make tiles of 16, 64 and 128
# rows of the batch, 80 of those sequences leave none divided.
BATCHES = {"alone": [1, 3], "in 64": [1, 3, 15, 2, 4], "in 128": [1, 200, 3, 4, 1], "whole": [40, 1, 2] * 28}


@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("softcap", [0.0, 8.0])
def test_short_sequences_keep_16_bits(softcap, d, cache, batch):
    """Queries of one element make scores one product each, so that little but the weights' own bits is rounded: a weight
    is cut to 8 bits and the rest, below 2^-7 of it, rounded to 8; 2^-20 of it is added.  A cap costs a tanh."""
    q_lens = BATCHES[batch]
    hk, group, ps = 16 if batch == "whole" else 2, 4, 16
    lens = [n + 150 + 13 * (i % 9) for i, n in enumerate(q_lens)]
    n_pages = max(-(-n // ps) for n in lens) + 2
    pages, scales, values = _cache(n_pages, ps, hk, d, cache, d)
    own = tables([max(lens)], ps, n_pages, n_pages, d)
    table = own.expand(len(lens), -1).contiguous()   # the sequences share their pages
    q = torch.zeros(sum(q_lens), hk * group, d)
    q.view(-1, d)[torch.arange(q.numel() // d), torch.arange(q.numel() // d) * 7 % d] = 1.0
    out = _run(q.to(BF16), q_lens, lens, table, pages, scales, hk, cache, scale=1.5, softcap=softcap)
    assert (out.abs() < 9).all()
    fine = coarse = 0
    first = 0
    for n, nk in zip(q_lens, lens):
        rows = slice(first, first + n)
        first += n
        if n * group > 16:
            continue
        for h in range(hk * group):
            k, v = (sequence64(values[x], own[0], nk, ps)[0][:, h // group] for x in "kv")
            s = 1.5 * q[rows, h].double() @ k.T
            err = 4 * U32 * s.abs().max()
            if softcap:
                s = softcap * torch.tanh(s / softcap)
                err = err + 2 * softcap * FN
            s[torch.arange(nk)[None] > nk - n + torch.arange(n)[:, None]] = -math.inf
            w = torch.softmax(s, 1)
            want, size = w @ v, w @ v.abs()
            bound = size * (2.0 ** -15 + 2.0 ** -20 + 2 * err + 2 * FN + 2 * nk * U32) + U * want.abs() + 1e-30
            assert ((out[rows, h] - want).abs() <= bound).all(), (n, nk, h, float(((out[rows, h] - want).abs() / bound).max()))
            # A weight of 8 bits would show: its output lies outside the bound somewhere.
            e = torch.exp(s)
            coarse += int(((e.float().to(BF16).double() @ v / e.sum(1, keepdim=True) - want).abs() > bound).sum())
            fine += want.numel()
    assert fine and (softcap or coarse > fine // 100)



@pytest.mark.parametrize("batch", ["alone", "in 64", "in 128", "whole"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_seen_infinities_of_short_sequences(value, d, batch):
    """An element among keys that every row sees, and one that the last row alone sees: they reach that element, with
    their sign, and no other."""
    q_lens = BATCHES[batch]
    hk, group, ps = 16 if batch == "whole" else 2, 4, 16
    lens = [n + 150 for n in q_lens]
    n_pages = max(-(-n // ps) for n in lens) + 2
    pages, scales, values = _cache(n_pages, ps, hk, d, "bf16", d)
    table = torch.arange(n_pages, dtype=torch.int32).expand(len(lens), -1).contiguous()
    short = [b for b, n in enumerate(q_lens) if 2 <= n <= 4][0]
    last = lens[short] - 1
    pages[1].view(-1, hk, d)[3, 0, 5] = value
    pages[1].view(-1, hk, d)[last, 1, d - 7] = value
    q = torch.zeros(sum(q_lens), hk * group, d)
    q.view(-1, d)[torch.arange(q.numel() // d), torch.arange(q.numel() // d) * 7 % d] = 1.0
    out = _run(q.to(BF16), q_lens, lens, table, pages, scales, hk, "bf16", scale=1.5)
    first = sum(q_lens[:short])
    for i in range(q_lens[short]):
        row, want = out[first + i], torch.zeros(hk * group, d, dtype=torch.float64)
        want[:group, 5] = value
        if i == q_lens[short] - 1:
            want[group:2 * group, d - 7] = value
        fine = torch.isfinite(want)
        assert torch.isfinite(row[fine]).all()
        assert torch.isnan(row[~fine]).all() if value != value else (row[~fine] == value).all()
