"""GPU: kv_cache_store and kv_cache_load against their definition, bit for bit: both types and caches, head sizes,
layouts, padding tokens, pages that are none, every code with every scale."""
import math

import pytest
import torch

from attention_reference import TYPES
from decoder_reference import E4M3, quantise64, random_cache, sequence64, tables

pytestmark = pytest.mark.gpu


def cc():
    import convolution_conv2d_forward_amd as m
    return m


def _empty_cache(n_pages, page_size, heads, d, dtype, cache):
    """Pages full of a pattern that shows what is written."""
    if cache != "e4m3":
        return [torch.full((n_pages, page_size, heads, d), 7.0, dtype=TYPES[dtype], device="cuda") for _ in "kv"] + [None] * 2
    pages = [torch.full((n_pages, page_size, heads, d), 0x55, dtype=torch.uint8, device="cuda").view(E4M3) for _ in "kv"]
    return pages + [torch.full((n_pages, page_size, heads), 99, dtype=torch.uint8, device="cuda") for _ in "kv"]


def _same(got, want):
    """Equal values, NaN in the same places."""
    got, want = got.cpu().double(), want.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, nan=0.0), torch.nan_to_num(want, nan=0.0))


def _check_store(k, v, slots, pages, heads, d, page_size, dtype, cache, **params):
    kp, vp, ks, vs = pages
    before = [None if t is None else t.cpu().clone() for t in pages]
    m = cc()
    desc = m.kv_cache_desc_create(m.make_kv_cache_params(heads, d, page_size, dtype=dtype, cache_dtype=cache,
                                                         k_stride=k.stride(0), v_stride=v.stride(0), **params))
    m.kv_cache_store(desc, k, v, torch.tensor(slots, dtype=torch.int32, device="cuda"), kp, vp, ks, vs)
    for x, p, s, p0, s0 in ((k, kp, ks, before[0], before[2]), (v, vp, vs, before[1], before[3])):
        want = p0.double()
        flags = torch.zeros(p.shape[:2], dtype=torch.bool)
        codes, e = quantise64(x.cpu()) if cache == "e4m3" else (x.cpu().double(), None)
        scales = None if s is None else s0.clone()
        for t, slot in enumerate(slots):
            if 0 <= slot < p.shape[0] * page_size:
                want[slot // page_size, slot % page_size] = codes[t]
                flags[slot // page_size, slot % page_size] = True
                if scales is not None:
                    scales[slot // page_size, slot % page_size] = (e[t] + 127).to(torch.uint8)
        _same(p, want)
        if s is not None:
            assert torch.equal(s.cpu(), scales)


@pytest.mark.parametrize("dtype,cache", [("bf16", "e4m3"), ("f32", "e4m3"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("heads,d", [(1, 1), (3, 8), (2, 20), (5, 33), (2, 64), (6, 80), (8, 128), (1, 136), (3, 250), (2, 256)])
@pytest.mark.parametrize("tokens,page_size", [(1, 1), (37, 5), (130, 16)])
def test_store(tokens, page_size, heads, d, dtype, cache):
    g = torch.Generator().manual_seed(tokens + d)
    n_pages = -(-tokens // page_size) + 3
    x = (torch.randn(2, tokens, heads, d, generator=g) * torch.exp(3 * torch.randn(2, tokens, heads, 1, generator=g))).to(TYPES[dtype]).cuda()
    slots = torch.randperm(n_pages * page_size, generator=g)[:tokens].tolist()
    if tokens > 8:   # padding tokens
        slots[3], slots[5], slots[7] = -1, n_pages * page_size, -2 ** 31
    _check_store(x[0], x[1], slots, _empty_cache(n_pages, page_size, heads, d, dtype, cache), heads, d, page_size, dtype, cache)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 20])
def test_store_values_at_the_borders(dtype, d):
    """Rows of zeros, of the type's smallest and largest numbers, maxima at 448 * 2^n and beside it, ties between codes,
    infinities and NaN."""
    t = TYPES[dtype]
    info = torch.finfo(t)
    rows = []
    one = torch.ones(d)
    for n in (-149, -140, -126, -118, -117, -110, -1, 0, 3, 100, 118, 119):
        for f in (448.0, 447.0, 449.0, 450.0, 1.0, 0.875, 0.8751):
            rows.append(one * f * 2.0 ** n if n > -127 else one * f * 2.0 ** -120 * 2.0 ** (n + 120))
    rows += [0 * one, -0.0 * one, info.max * one, info.min * one, info.tiny * one, one * 1.5 * info.tiny]
    ties = torch.linspace(-448, 448, 2 * d - 1)[:d]
    rows += [ties, torch.arange(d) * 2.0 ** -10, torch.arange(d) * 2.0 ** -9 + 2.0 ** -10]
    rows += [torch.where(torch.arange(d) == 0, 448.0, (8.0 + torch.arange(d) % 8 + 0.5) * 2.0 ** (torch.arange(d) % 9 - 8))]
    for bad in (math.inf, -math.inf, math.nan):
        r = torch.randn(d, generator=torch.Generator().manual_seed(1))
        r[1] = bad
        rows += [r, one * bad]
    x = torch.stack(rows).to(t)[:, None].cuda()
    n = x.shape[0]
    _check_store(x, -x, list(range(n)), _empty_cache(-(-n // 16), 16, 1, d, dtype, "e4m3"), 1, d, 16, dtype, "e4m3")


@pytest.mark.parametrize("dtype,cache", [("bf16", "e4m3"), ("f32", "f32")])
@pytest.mark.parametrize("d", [64, 36])
def test_layouts(d, dtype, cache):
    """Values inside a projection's rows; keys and values of a page beside each other; heads before tokens."""
    heads, tokens, ps, n_pages, t = 3, 50, 8, 9, TYPES[dtype]
    g = torch.Generator().manual_seed(d)
    qkv = torch.randn(tokens, 5 * heads, d, generator=g).to(t).cuda()
    k, v = qkv[:, 3 * heads:4 * heads], qkv[:, 4 * heads:]
    slots = torch.randperm(n_pages * ps, generator=g)[:tokens].tolist()
    ct = torch.uint8 if cache == "e4m3" else t
    wide = torch.zeros(n_pages, 2, ps, heads, d, dtype=ct, device="cuda")
    wide = wide.view(E4M3) if cache == "e4m3" else wide
    scales = [torch.zeros(n_pages, ps, heads, dtype=torch.uint8, device="cuda") for _ in "kv"] if cache == "e4m3" else [None] * 2
    both = [wide[:, 0], wide[:, 1]] + scales
    strides = dict(k_page_strides=both[0].stride()[:3], v_page_strides=both[1].stride()[:3])
    _check_store(k, v, slots, both, heads, d, ps, dtype, cache, **strides)
    turned = [torch.zeros(n_pages, heads, ps, d, dtype=ct, device="cuda") for _ in "kv"]
    turned = [(x.view(E4M3) if cache == "e4m3" else x).transpose(1, 2) for x in turned]
    if cache == "e4m3":
        scales = [torch.zeros(n_pages, heads, ps, dtype=torch.uint8, device="cuda").transpose(1, 2) for _ in "kv"]
        strides["scale_strides"] = scales[0].stride()
    strides.update(k_page_strides=turned[0].stride()[:3], v_page_strides=turned[1].stride()[:3])
    _check_store(k, v, slots, turned + scales, heads, d, ps, dtype, cache, **strides)
    # Back, into rows of a larger buffer.
    m = cc()
    table = torch.tensor([[4, 0, 8], [1, 7, 2]], dtype=torch.int32)
    out = torch.full((2, 30, 2 * heads, d), 5.0, dtype=t, device="cuda")
    desc = m.kv_cache_desc_create(m.make_kv_cache_params(
        heads, d, ps, dtype=dtype, cache_dtype=cache, k_stride=out.stride(1), v_stride=out.stride(1), **strides))
    m.kv_cache_load(desc, table.cuda(), torch.tensor([24, 9], dtype=torch.int32, device="cuda"), turned[0], turned[1],
                    *scales, out[:, :, :heads], out[:, :, heads:])
    for n, x, s, at in (("k", turned[0], scales[0], 0), ("v", turned[1], scales[1], heads)):
        values = x.cpu().double()
        if s is not None:
            values = torch.ldexp(values, s.cpu().to(torch.int32)[..., None] - 127)
        for b, length in enumerate((24, 9)):
            _same(out[b, :length, at:at + heads], sequence64(values, table[b], length, ps)[0])
            assert (out[b, length:, at:at + heads] == 5).all()


@pytest.mark.parametrize("dtype,cache", [("bf16", "e4m3"), ("f32", "e4m3"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("heads,d", [(1, 1), (2, 20), (5, 33), (2, 64), (6, 80), (8, 128), (2, 256)])
@pytest.mark.parametrize("page_size", [1, 7, 16])
def test_load(page_size, heads, d, dtype, cache):
    """Lengths of zero, one, beyond the buffer and the table; a page that is none leaves its rows."""
    t, max_pages, kv_len = TYPES[dtype], -(-60 // page_size), 53
    lens = [53, 0, 1, 60, 17, -3]
    n_pages = sum(-(-max(n, 0) // page_size) for n in lens) + 2
    got, values = random_cache(n_pages, page_size, heads, d, dtype, cache, seed=d)
    table = tables(lens, page_size, n_pages, max_pages)
    table[4, 1 % max_pages] = n_pages
    table[0, 0] = -7
    k, v = (torch.full((len(lens), kv_len, heads, d), 5.0, dtype=t, device="cuda") for _ in "kv")
    m = cc()
    desc = m.kv_cache_desc_create(m.make_kv_cache_params(heads, d, page_size, dtype=dtype, cache_dtype=cache))
    dev = [None if got[n] is None else got[n].cuda() for n in ("k", "v", "ks", "vs")]
    m.kv_cache_load(desc, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), *dev, k, v)
    for n, out in (("k", k), ("v", v)):
        for b, length in enumerate(lens):
            length = min(max(length, 0), kv_len)
            want, there = sequence64(values[n], table[b], length, page_size)
            _same(out[b, :length], torch.where(there[:, None, None], want, 5.0))
            assert (out[b, length:] == 5).all()
    m.kv_cache_load(desc, table.cuda(), None, *dev, k, v)
    want, there = sequence64(values["k"], table[3], kv_len, page_size)
    _same(k[3], want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [128, 31])
def test_every_code_with_every_scale(dtype, d):
    """Each code times each power is exact in both types."""
    n = -(-256 // d)
    codes = (torch.arange(n * d) % 256).to(torch.uint8).view(1, 1, n, d).expand(1, 237, n, d).contiguous()
    scales = torch.arange(10, 247).to(torch.uint8).view(1, 237, 1).expand(1, 237, n).contiguous()
    m = cc()
    desc = m.kv_cache_desc_create(m.make_kv_cache_params(n, d, 237, dtype=dtype, cache_dtype="e4m3"))
    k, v = (torch.zeros(1, 237, n, d, dtype=TYPES[dtype], device="cuda") for _ in "kv")
    pages, s = codes.view(E4M3).cuda(), scales.cuda()
    m.kv_cache_load(desc, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), None, pages, pages, s, s, k, v)
    want = torch.ldexp(codes.view(E4M3).double(), scales.to(torch.int32)[..., None] - 127)
    _same(k, want)
    _same(v, want)


def test_nothing_to_do():
    m = cc()
    desc = m.kv_cache_desc_create(m.make_kv_cache_params(2, 8, 4, dtype="bf16", cache_dtype="e4m3"))
    new = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    none = torch.zeros(0, 4, 2, 8, dtype=torch.uint8, device="cuda").view(E4M3)
    s = torch.zeros(0, 4, 2, dtype=torch.uint8, device="cuda")
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    m.kv_cache_store(desc, new(0, 2, 8), new(0, 2, 8), ints(), none, none, s, s)
    m.kv_cache_store(desc, new(1, 2, 8), new(1, 2, 8), ints(0), none, none, s, s)
    out = new(1, 5, 2, 8) + 3
    m.kv_cache_load(desc, ints(0, 1).view(1, 2), None, none, none, s, s, out, new(1, 5, 2, 8))
    assert (out == 3).all()


def test_pages_beyond_32_bit_offsets():
    """Pages 2^31 elements apart, and a slot number of the last one."""
    heads, d, ps, n_pages = 2, 64, 4, 3
    stride = 1 << 31
    m = cc()
    buf = [torch.zeros((n_pages - 1) * stride + ps * heads * d, dtype=torch.uint8, device="cuda") for _ in "kv"]
    pages = [b.view(E4M3).as_strided((n_pages, ps, heads, d), (stride, heads * d, d, 1)) for b in buf]
    scales = [torch.zeros(n_pages, ps, heads, dtype=torch.uint8, device="cuda") for _ in "kv"]
    strides = dict(k_page_strides=pages[0].stride()[:3], v_page_strides=pages[1].stride()[:3])
    desc = m.kv_cache_desc_create(m.make_kv_cache_params(heads, d, ps, dtype="bf16", cache_dtype="e4m3", **strides))
    x = torch.randn(2, 5, heads, d, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    slots = [11, 8, 4, 0, 9]
    m.kv_cache_store(desc, x[0].cuda(), x[1].cuda(), torch.tensor(slots, dtype=torch.int32, device="cuda"), *pages, *scales)
    k, v = (torch.zeros(1, 12, heads, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    m.kv_cache_load(desc, torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"), None, *pages, *scales, k, v)
    for got, src in ((k, x[0]), (v, x[1])):
        codes, e = quantise64(src)
        for t, slot in enumerate(slots):
            _same(got[0, slot], torch.ldexp(codes[t], e[t][:, None]))


@pytest.mark.parametrize("d", [8, 256, 5])
def test_many_heads(d):
    """As many heads as a descriptor takes, stored and brought back as they are."""
    m, heads, ps = cc(), 1 << 16, 2
    desc = m.kv_cache_desc_create(m.make_kv_cache_params(heads, d, ps, dtype="bf16"))
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn(3, heads, d, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv")
    pages = [torch.zeros(3, ps, heads, d, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    m.kv_cache_store(desc, k, v, ints([5, 0, 4]), *pages)
    out = [torch.zeros(2, 3, heads, d, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    m.kv_cache_load(desc, ints([[2, 0], [0, 3]]), ints([3, 4]), *pages, None, None, *out)
    for x, page, y in zip((k, v), pages, out):
        assert torch.equal(page.view(6, heads, d)[[5, 0, 4]], x) and not page.view(6, heads, d)[[1, 2, 3]].any()
        assert torch.equal(y[0], x[[2, 0, 1]]) and torch.equal(y[1, 0], x[1]) and not y[1, 1:].any()
