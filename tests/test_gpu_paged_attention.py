"""GPU: paged_attention_forward against the 64-bit definition: single tokens, chunks and both in a batch, every cache
type, pages of any size, windows with first tokens, rows that see nothing, garbage where no row looks."""
import pytest
import torch

from attention_reference import TYPES, assert_within
from decoder_reference import paged64, random_cache, tables

pytestmark = pytest.mark.gpu

KINDS = [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32"), ("f32", "e4m3")]


def cc():
    import convolution_conv2d_forward_amd as m
    return m


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _offsets(q_lens, first=0):
    return [first + sum(q_lens[:i]) for i in range(len(q_lens) + 1)]


def _desc(hq, hk, d, ps, c, **strides):
    m = cc()
    return m.paged_attention_desc_create(m.make_paged_attention_params(
        hq, hk, d, ps, window=c.get("window", 0), sinks=c.get("sinks", 0), softcap=c.get("softcap", 0.0),
        scale=c.get("scale"), dtype=c["dtype"], cache_dtype=c["cache"], **strides))


def _run(desc, q, offsets, lens, table, cache, out=None, stream=None):
    """Device tensors but for the lists; out is filled with 9 before."""
    m = cc()
    if out is None:
        out = torch.full(q.shape, 9.0, dtype=q.dtype, device="cuda")
    n = m.paged_attention_workspace_bytes(desc, q.shape[0], table.shape[0], table.shape[1])
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None
    m.paged_attention_forward(desc, q, _ints(offsets), _ints(lens), table, *cache, out, workspace=ws, stream=stream)
    return out


def _check(q_lens, kv_lens, hq, hk, d, ps, dtype, cache, seed=0, first=0, extra=0, change=None, spare=2, sharp=2.0, **c):
    c.update(dtype=dtype, cache=cache)
    clean = [max(n, 0) for n in kv_lens]
    max_pages = max(1, -(-max(clean) // ps))
    n_pages = sum(-(-n // ps) for n in clean) + spare
    got, values = random_cache(n_pages, ps, hk, d, dtype, cache, seed + 1)
    table = tables(clean, ps, n_pages, max_pages, seed)
    offsets = _offsets(q_lens, first)
    tokens = offsets[-1] + extra
    g = torch.Generator().manual_seed(seed)
    q = (sharp * torch.randn(tokens, hq, d, generator=g)).to(TYPES[dtype])
    if change:
        change(table, got, values)
    dev = [None if got[n] is None else got[n].cuda() for n in ("k", "v", "ks", "vs")]
    out = _run(_desc(hq, hk, d, ps, c), q.cuda(), offsets, kv_lens, table.cuda(), dev)
    want, tol, mine = paged64(q, offsets, kv_lens, table, values, c)
    want[~mine], tol[~mine] = 9.0, 0.0
    assert_within(out, want, tol, f"{q_lens} {kv_lens} {hq}/{hk} d{d} page {ps} {c}")
    return out


DIMS = {"bf16": [8, 24, 32, 64, 72, 80, 96, 128, 136, 200, 256], "f32": [4, 20, 32, 64, 96, 100, 128, 160, 256]}


@pytest.mark.parametrize("dtype,cache,d", [(t, c, d) for t, c in KINDS for d in DIMS[t] if c == t or d % 16 == 0])
@pytest.mark.parametrize("q_len", [1, 9, 70])
def test_head_dims(q_len, dtype, cache, d):
    _check([q_len, q_len - 1], [150, 131], 4, 2, d, 16, dtype, cache, seed=d, softcap=30.0)


LENGTHS = [(1, 1), (1, 2), (1, 31), (1, 33), (1, 64), (1, 257), (1, 1100), (2, 2), (3, 500), (5, 17), (8, 1030), (16, 16),
           (17, 900), (33, 70), (64, 64), (65, 130), (127, 127), (129, 129), (200, 333), (300, 300), (7, 3), (1, 0), (40, 12)]


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("q_len,kv_len", LENGTHS)
def test_lengths(q_len, kv_len, dtype, cache):
    """(7, 3), (40, 12): the first rows are before every key."""
    _check([q_len], [kv_len], 4, 1, 64, 16, dtype, cache, seed=q_len + kv_len)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("ps", [1, 2, 7, 16, 20, 48, 64, 100, 256])
@pytest.mark.parametrize("q_len", [1, 50])
def test_page_sizes(q_len, ps, dtype, cache):
    _check([q_len, 1, q_len], [211, 64, 130], 4, 2, 64, ps, dtype, cache, seed=ps)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (6, 2), (5, 1), (16, 1), (32, 4), (24, 1)])
@pytest.mark.parametrize("q_len", [1, 4, 50])
def test_groups(q_len, hq, hk, dtype, cache):
    _check([q_len, 1], [90, 77], hq, hk, 128, 16, dtype, cache, seed=hq)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("q_len,kv_len", [(1, 400), (6, 300), (180, 180), (140, 400)])
@pytest.mark.parametrize("c", [
    dict(softcap=20.0), dict(window=1), dict(window=1, sinks=1), dict(window=40), dict(window=40, sinks=4),
    dict(window=65, sinks=64), dict(window=30, sinks=100), dict(window=2 ** 31 - 1, sinks=3),
    dict(window=100, sinks=2 ** 31 - 1), dict(sinks=5), dict(window=64, sinks=65, softcap=8.0), dict(scale=0.5),
    dict(scale=-0.3, window=50, sinks=2), dict(scale=0.0, window=50), dict(softcap=1000.0), dict(scale=-0.2, softcap=9.0),
], ids=lambda c: "-".join("%s%g" % i for i in c.items()))
def test_masks_and_caps(c, q_len, kv_len, dtype, cache):
    _check([q_len, min(q_len, 3)], [kv_len, kv_len - 61], 4, 2, 64, 16, dtype, cache, seed=7, **c)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("c", [{}, dict(window=70, sinks=5), dict(softcap=15.0)], ids=str)
def test_batches_of_all_kinds(c, dtype, cache):
    """Chunks among single tokens, sequences without new ones, without keys, with lengths beyond the table; rows before
    the first and behind the last sequence stay as they were."""
    _check([1, 100, 0, 1, 1, 37, 1, 3, 0], [500, 300, 40, 0, 1, 37, 90, 2, 0], 8, 2, 64, 16, dtype, cache, seed=3,
           first=5, extra=11, **c)
    _check([2, 1], [100, 77], 4, 4, 128, 8, dtype, cache, first=1, extra=1, change=lambda t, *_: None, **c)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("q_lens", [[1] * 5, [60, 1, 33, 1, 2]], ids=str)
def test_lengths_beyond_the_table_and_below_zero(q_lens, dtype, cache):
    c = dict(dtype=dtype, cache=cache)
    got, values = random_cache(20, 16, 2, 64, dtype, cache)
    table = tables([64] * 5, 16, 20, 4)
    lens = [65, -1, 10 ** 9, 64, -2 ** 31]
    q = torch.randn(sum(q_lens), 4, 64).to(TYPES[dtype])
    dev = [None if got[n] is None else got[n].cuda() for n in ("k", "v", "ks", "vs")]
    out = _run(_desc(4, 2, 64, 16, c), q.cuda(), _offsets(q_lens), lens, table.cuda(), dev)
    want, tol, _ = paged64(q, _offsets(q_lens), lens, table, values, c)
    assert_within(out, want, tol)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [200, 150, 90]), ([130, 1, 64], [200, 150, 90])], ids=str)
@pytest.mark.parametrize("ps", [4, 16, 64])
def test_bad_pages(ps, q_lens, kv_lens, dtype, cache):
    """Keys on pages that are none are seen by no row: single ones, a whole sequence's."""
    def change(table, got, values):
        n = values["k"].shape[0]
        table[0, 0], table[0, 1], table[1, table.shape[1] // 2] = -1, n, -2 ** 31
        table[0, 2] = 2 ** 31 - 1
        table[2] = n + 5
    _check(q_lens, kv_lens, 4, 2, 64, ps, dtype, cache, change=change)
    _check(q_lens, kv_lens, 4, 2, 128, ps, dtype, cache, change=change, window=60, sinks=20)


def test_no_pages_and_nothing_to_do():
    c = dict(dtype="bf16", cache="bf16")
    new = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, d = new(3, 4, 64) + 1, _desc(4, 2, 64, 16, c)
    for n_pages, max_pages in ((0, 2), (1, 0), (0, 0)):
        out = _run(d, q, [0, 1, 3], [20, 20], torch.zeros(2, max_pages, dtype=torch.int32, device="cuda"),
                   [new(n_pages, 16, 2, 64), new(n_pages, 16, 2, 64), None, None])
        assert (out == 0).all()
    out = _run(d, q, [0], [], torch.zeros(0, 2, dtype=torch.int32, device="cuda"), [new(1, 16, 2, 64)] * 2 + [None] * 2)
    assert (out == 9).all()
    _run(d, q[:0], [0, 0], [5], torch.zeros(1, 2, dtype=torch.int32, device="cuda"), [new(1, 16, 2, 64)] * 2 + [None] * 2)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("q_len,kv_len", [(1, 200), (3, 600), (150, 150), (90, 280)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_unseen_garbage_does_not_spread(bad, q_len, kv_len, dtype, cache):
    """Infinities and NaN in the tail of a last page, on pages of no sequence, in the future of rows and outside the
    window; the rows that see one get it."""
    def change(table, got, values):
        quantised = cache == "e4m3"

        def put(n, page, token, head=slice(None), e=slice(None)):
            value = float("nan") if quantised else bad
            if quantised:
                got[n].view(torch.uint8)[page, token, head, e] = 0x7f if bad > 0 else 0xff
            else:
                got[n][page, token, head, e] = bad
            values[n][page, token, head, e] = value
        used = set(int(p) for p in table.flatten() if p >= 0)
        for page in range(values["k"].shape[0]):
            if page not in used:
                put("k", page, slice(None))
                put("v", page, slice(None))
        at = lambda b, j: (int(table[b, j // 16]), j % 16)  # noqa: E731
        for b, n in ((0, kv_len), (1, kv_len - 25)):
            page, token = at(b, n - 1)
            for t in range(token + 1, 16):   # behind the sequence's end
                put("k", page, t)
                put("v", page, t)
            if quantised:   # scale bytes that nobody wrote
                got["ks"][page, token + 1:], got["vs"][page, token + 1:] = 255, 0
                got["vs"][page, token + 2:] = 254
        put("v", *at(0, kv_len - 1), 0, 3)   # the last key: seen by the last row alone
        put("v", *at(0, kv_len // 2), 1, 7)
        put("v", *at(1, 2), 1, 9)            # one of the first tokens
        if bad != bad:
            put("k", *at(0, 20))
    _check([q_len, 1], [kv_len, kv_len - 25], 4, 2, 64, 16, dtype, cache, seed=4, change=change, spare=3, window=60, sinks=4)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("q_len", [1, 70])
def test_layouts(q_len, dtype, cache):
    """Queries inside a projection's rows, out in a wider buffer; keys and values of a page in one buffer; heads before
    tokens; scales alike."""
    c = dict(dtype=dtype, cache=cache, window=90, sinks=3)
    hq, hk, d, ps, lens = 6, 3, 64, 8, [100, 61]
    got, values = random_cache(24, ps, hk, d, dtype, cache, 5)
    table = tables(lens, ps, 24, 13)
    tokens = q_len + 1
    qkv = torch.randn(tokens, hq + 2 * hk, d, generator=torch.Generator().manual_seed(2)).to(TYPES[dtype])
    want, tol, _ = paged64(qkv[:, :hq], [0, q_len, tokens], lens, table, values, c)
    raw = lambda t: t.view(torch.uint8) if cache == "e4m3" else t  # noqa: E731
    pair = raw(torch.stack([raw(got["k"]), raw(got["v"])], 1)).cuda()
    pair = pair.view(got["k"].dtype)
    heads = [raw(got[n]).transpose(1, 2).contiguous().cuda().view(got[n].dtype).transpose(1, 2) for n in "kv"]
    scales = [None, None] if cache != "e4m3" else [got["ks"].cuda(), got["vs"].cuda()]
    turned = [None if s is None else s.transpose(1, 2).contiguous().transpose(1, 2) for s in scales]
    for k, v, s in ((pair[:, 0], pair[:, 1], scales), (heads[0], heads[1], turned)):
        q, wide = qkv.cuda()[:, :hq], torch.full((tokens, 2 * hq, d), 9.0, dtype=TYPES[dtype], device="cuda")
        out = wide[:, hq:]
        strides = dict(q_stride=q.stride(0), out_stride=out.stride(0), k_page_strides=k.stride()[:3],
                       v_page_strides=v.stride()[:3])
        if s[0] is not None:
            strides["scale_strides"] = s[0].stride()
        _run(_desc(hq, hk, d, ps, c, **strides), q, [0, q_len, tokens], lens, table.cuda(), [k, v] + s, out)
        assert_within(out, want, tol)
        assert (wide[:, :hq] == 9).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_len", [1, 40])
def test_pages_beyond_32_bit_offsets(q_len, cache):
    """Pages 2^30 elements (2^31 of them E4M3) apart."""
    c = dict(dtype="bf16", cache=cache)
    hk, d, ps, lens = 2, 64, 16, [44]
    got, values = random_cache(3, ps, hk, d, "bf16", cache, 6)
    far = 1 << (30 if cache == "bf16" else 31)
    pages = []
    for n in "kv":
        buf = torch.zeros(2 * far + ps * hk * d, dtype=torch.uint8 if cache == "e4m3" else torch.bfloat16, device="cuda")
        at = buf.view(got[n].dtype).as_strided((3, ps, hk, d), (far, hk * d, d, 1))
        buf.as_strided((3, ps, hk, d), (far, hk * d, d, 1)).copy_(got[n].view(buf.dtype))
        pages.append(at)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    q = torch.randn(q_len, 4, d, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    desc = _desc(4, hk, d, ps, c, k_page_strides=pages[0].stride()[:3], v_page_strides=pages[1].stride()[:3])
    scales = [None, None] if cache == "bf16" else [got["ks"].cuda(), got["vs"].cuda()]
    out = _run(desc, q.cuda(), [0, q_len], lens, table.cuda(), pages + scales)
    want, tol, _ = paged64(q, [0, q_len], lens, table, values, c)
    assert_within(out, want, tol)


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_long_caches_and_same_results_twice(dtype, cache):
    """Keys divided among workgroups, sequences of very different length; a page shared by two sequences."""
    c = dict(dtype=dtype, cache=cache, softcap=50.0)
    lens, ps = [9000, 1, 4097, 333], 64
    got, values = random_cache(250, ps, 2, 128, dtype, cache, 11)
    table = tables(lens, ps, 250, 150)
    table[2, :30] = table[0, :30]
    q_lens = [1, 1, 2, 1]
    q = (2 * torch.randn(5, 8, 128, generator=torch.Generator().manual_seed(1))).to(TYPES[dtype])
    dev = [None if got[n] is None else got[n].cuda() for n in ("k", "v", "ks", "vs")]
    desc = _desc(8, 2, 128, ps, c)
    out = _run(desc, q.cuda(), _offsets(q_lens), lens, table.cuda(), dev)
    want, tol, _ = paged64(q, _offsets(q_lens), lens, table, values, c)
    assert_within(out, want, tol)
    assert torch.equal(out, _run(desc, q.cuda(), _offsets(q_lens), lens, table.cuda(), dev))
    q = (2 * torch.randn(151, 8, 128, generator=torch.Generator().manual_seed(2))).to(TYPES[dtype])
    q_lens = [100, 1, 50, 0]
    out = _run(desc, q.cuda(), _offsets(q_lens), lens, table.cuda(), dev)
    want, tol, _ = paged64(q, _offsets(q_lens), lens, table, values, c)
    assert_within(out, want, tol)
    assert torch.equal(out, _run(desc, q.cuda(), _offsets(q_lens), lens, table.cuda(), dev))


@pytest.mark.parametrize("cache,d", [("bf16", 8), ("e4m3", 16)])
@pytest.mark.parametrize("q_len,tol", [(1, 2.0 ** -6), (20, 2.0 ** -4)])
def test_keys_up_to_the_limit(q_len, tol, cache, d):
    """2^30 keys, one page over and over: what attention over that page gives (the last new tokens, which see a few keys
    less, too).  A lane adds up to 2^17 weights (single tokens) or 2^18.5 (chunks) in fp32, and as many products: each
    addition is off by 2^-24 of the sum, twice."""
    ps = 4096
    got, values = random_cache(2, ps, 1, d, "bf16", cache, 5)
    table = torch.ones(1, (1 << 30) // ps, dtype=torch.int32)
    q = torch.randn(q_len, 1, d, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    dev = [None if got[n] is None else got[n].cuda() for n in ("k", "v", "ks", "vs")]
    out = _run(_desc(1, 1, d, ps, dict(dtype="bf16", cache=cache)), q.cuda(), [0, q_len], [1 << 30], table.cuda(), dev)
    k, v = values["k"][1, :, 0], values["v"][1, :, 0]
    w = torch.softmax(d ** -0.5 * q[:, 0].double() @ k.T, 1)
    bound = tol * (w @ v.abs()) + 2.0 ** -7 * (w @ v.abs())   # the weights' and the output's own rounding
    assert ((out[:, 0].double().cpu() - w @ v).abs() <= bound).all()


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("batch", [70, 1100])
def test_many_sequences(batch, dtype, cache):
    lens = [(37 * i) % 90 for i in range(batch)]
    q_lens = [1 + 2 * (i % 11 == 3) if i % 5 else 0 for i in range(batch)]
    _check(q_lens, lens, 2, 1, 32, 16, dtype, cache)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("q_len,batch,heads", [(40, 36, 32), (40, 80, 16), (100, 30, 36), (1, 80, 32)])
def test_enough_rows_for_whole_tiles(q_len, batch, heads, dtype, cache):
    """Two rounds of workgroups and more: no tile is divided."""
    lens = [(37 * i) % 90 + q_len // 2 for i in range(batch)]
    _check([q_len - i % 3 if q_len > 1 else 1 for i in range(batch)], lens, heads, heads, 32, 16, dtype, cache)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("c", [{}, dict(window=200, sinks=70)], ids=str)
@pytest.mark.parametrize("q_lens", [[900, 40, 1], [0, 700, 3]], ids=str)
def test_more_tiles_than_lanes(q_lens, c, dtype, cache):
    """Tiles of a few sequences that are more than 64, and divided."""
    _check(q_lens, [1000, 700, 90], 24, 2, 32, 16, dtype, cache, **c)


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_large_scores(dtype, cache):
    """Scores of thousands: weights of 0 and 1, no overflow; scores all equal to a large negative number."""
    out = _check([40, 1], [200, 200], 2, 1, 64, 16, dtype, cache, sharp=0.0)
    for sharp in (300.0, -300.0):
        c = dict(dtype=dtype, cache=cache)
        got, values = random_cache(13, 16, 1, 64, dtype, cache)
        q = (sharp * torch.randn(40, 2, 64, generator=torch.Generator().manual_seed(4))).to(TYPES[dtype])
        dev = [None if got[n] is None else got[n].cuda() for n in ("k", "v", "ks", "vs")]
        out = _run(_desc(2, 1, 64, 16, c), q.cuda(), [0, 40], [200], torch.arange(13, dtype=torch.int32).cuda()[None], dev)
        assert torch.isfinite(out).all()
        assert (out.double().abs() <= values["v"].abs().max().cuda() * (1 + 2.0 ** -7)).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_captured_steps_and_another_stream(cache):
    """One captured call replayed over changed lengths, tables and queries, other work between; a call on a side stream."""
    m = cc()
    c = dict(dtype="bf16", cache=cache, window=300, sinks=4)
    ps, lens = 16, [400, 90, 650]
    got, values = random_cache(90, ps, 2, 64, "bf16", cache, 3)
    dev = [None if got[n] is None else got[n].cuda() for n in ("k", "v", "ks", "vs")]
    desc = _desc(4, 2, 64, ps, c)
    table = tables(lens, ps, 90, 41)
    q, out = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    off, kv, tab = _ints([0, 1, 2, 3]), _ints(lens), table.cuda()
    n = m.paged_attention_workspace_bytes(desc, 3, 3, 41)
    ws = torch.zeros(max(n, 1), dtype=torch.uint8, device="cuda")
    call = lambda: m.paged_attention_forward(desc, q, off, kv, tab, *dev, out, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    g = torch.Generator().manual_seed(9)
    for step in range(4):
        x = torch.randn(3, 4, 64, generator=g).to(torch.bfloat16)
        now = [max(1, length - 97 * step) for length in lens]
        other = table.flip(0) if step % 2 else table
        now = now[::-1] if step % 2 else now
        q.copy_(x)
        kv.copy_(torch.tensor(now, dtype=torch.int32))
        tab.copy_(other)
        out.fill_(float("nan"))
        graph.replay()
        want, tol, _ = paged64(x, [0, 1, 2, 3], now, other, values, c)
        assert_within(out, want, tol, f"replay {step}")
        torch.cuda.synchronize()
    out.fill_(float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    m.paged_attention_forward(desc, q, off, kv, tab, *dev, out, workspace=ws, stream=side)
    side.synchronize()
    assert_within(out, want, tol)
