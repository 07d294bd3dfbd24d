"""GPU: the paged cache, attention over it and block_norm together, captured and replayed, on other streams, and with one
workspace between two graphs."""
import os
import sys

import pytest
import torch

from attention_reference import TYPES, assert_within
from decoder_reference import paged64, random_cache, tables
from test_gpu_paged_attention import _desc, _ints, _offsets, _run

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def cc():
    import convolution_conv2d_forward_amd as m
    return m


# An output passes some 20 roundings in two layers, by either way: that many half-steps (bf16 2^-9 to 2^-8, fp32 2^-25 to
# 2^-24, and fp32 sums of 1024 terms beside) on the largest output stay below these.
@pytest.mark.parametrize("dtype,cache,tol", [("bf16", "e4m3", 2.0 ** -4), ("bf16", "bf16", 2.0 ** -4),
                                             ("f32", "e4m3", 2.0 ** -14), ("f32", "f32", 2.0 ** -14)])
@pytest.mark.parametrize("c", [{}, dict(window=100), dict(head_dim=128, heads_q=4, heads_kv=1, page_size=7)], ids=str)
def test_example_steps_match_rows_brought_back(c, dtype, cache, tol):
    """Prompts in ragged chunks, captured single tokens, and the same tokens by kv_cache_load and attention_forward."""
    import paged_decoder
    got, again, _ = paged_decoder.run(lens=(300, 40, 1, 129), chunk=100, steps=5, width=256, hidden=512, dtype=dtype,
                                      cache=cache, **c)
    assert torch.isfinite(got).all() and torch.isfinite(again).all()
    assert float((got.double() - again.double()).abs().max()) <= tol * float(again.abs().max())


def test_example_with_first_tokens_kept():
    import paged_decoder
    got, again, _ = paged_decoder.run(lens=(300, 40, 1), chunk=100, steps=5, width=256, hidden=512, window=64, sinks=4)
    assert again is None and torch.isfinite(got).all()
    whole, _, _ = paged_decoder.run(lens=(300, 40, 1), chunk=100, steps=5, width=256, hidden=512, window=64)
    near = lambda i: float((got[i] - whole[i]).abs().max()) <= 2.0 ** -4 * float(whole.abs().max())  # noqa: E731
    assert near(1) and near(2)   # up to 45 tokens: all within the window, the keys divided elsewhere
    assert not torch.equal(got[0], whole[0])


def _captured(call):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    return graph


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,d", [(2, 64), (3, 24)])
def test_store_and_load_captured(heads, d, cache):
    """A graph of a store and a load, replayed over other rows, slots, tables and lengths, work between: as eager calls."""
    m, ps, n_pages, g = cc(), 8, 30, torch.Generator().manual_seed(0)
    desc = m.kv_cache_desc_create(m.make_kv_cache_params(heads, d, ps, dtype="bf16", cache_dtype=cache))
    t = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16

    def pages():
        got = [torch.zeros((n_pages, ps, heads, d), dtype=torch.uint8 if cache == "e4m3" else t, device="cuda").view(t)
               for _ in "kv"]
        return got + [torch.full((n_pages, ps, heads), 127, dtype=torch.uint8, device="cuda") if cache == "e4m3" else None
                      for _ in "kv"]
    k, v = (torch.zeros(40, heads, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    slots, table, lens = _ints([-1] * 40), _ints([[0] * 6] * 3), _ints([0] * 3)

    def out():
        return [torch.zeros(3, 45, heads, d, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    a, b, rows_a, rows_b = pages(), pages(), out(), out()

    def call(got, rows, **kw):
        m.kv_cache_store(desc, k, v, slots, *got, **kw)
        m.kv_cache_load(desc, table, lens, *got, *rows, **kw)
    graph = _captured(lambda: call(a, rows_a))
    side = torch.cuda.Stream()
    for step in range(4):
        for x in (k, v):
            x.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))
        slots.copy_(torch.randperm(n_pages * ps, generator=g)[:40].to(torch.int32) - 20)
        table.copy_(torch.randint(-1, n_pages + 1, (3, 6), generator=g).to(torch.int32))
        lens.copy_(torch.tensor([45, 7 * step, 60], dtype=torch.int32))
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        call(b, rows_b, stream=side)
        torch.cuda.synchronize()
        for x, y in zip(a + rows_a, b + rows_b):
            assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8)), step
    assert float(rows_a[0].float().abs().max()) > 1


@pytest.mark.parametrize("width", [256, 513, 9001])
def test_norm_captured(width):
    m, rows, g = cc(), 37, torch.Generator().manual_seed(1)
    desc = m.block_norm_desc_create(m.make_block_norm_params(width, post_norm="rms", pre_norm="layer", dtype="bf16"))
    y, x, r, o = (torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    gammas = [torch.randn(width, generator=g).cuda() for _ in range(2)]
    call = lambda r, o, **kw: m.block_norm_forward(desc, y, x, None, gammas[0], None, gammas[1], None, r, o, **kw)  # noqa: E731
    graph, side = _captured(lambda: call(r, o)), torch.cuda.Stream()
    for step in range(4):
        for t in (x, y):
            t.copy_(torch.randn(t.shape, generator=g).to(torch.bfloat16))
        graph.replay()
        want = [torch.empty_like(r), torch.empty_like(o)]
        side.wait_stream(torch.cuda.current_stream())
        call(*want, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(r, want[0]) and torch.equal(o, want[1]), step


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_two_graphs_share_a_workspace(cache):
    """Single tokens and a chunk, captured over one workspace and replayed in turn on one stream."""
    m, ps, c = cc(), 16, dict(dtype="bf16", cache=cache)
    lens = [500, 900]
    got, values = random_cache(100, ps, 2, 64, "bf16", cache, 3)
    dev = [None if got[n] is None else got[n].cuda() for n in ("k", "v", "ks", "vs")]
    table, desc = tables(lens, ps, 100, 60), _desc(8, 2, 64, ps, c)
    calls = []
    for q_lens in ([1, 1], [70, 40]):
        q = torch.randn(sum(q_lens), 8, 64, generator=torch.Generator().manual_seed(len(calls))).to(torch.bfloat16)
        calls.append((q_lens, q, q.cuda(), torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda"), _ints(_offsets(q_lens))))
    need = max(m.paged_attention_workspace_bytes(desc, sum(n), 2, 60) for n, *_ in calls)
    assert need > 0
    ws, kv, tab = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda"), _ints(lens), table.cuda()
    graphs = [_captured(lambda q=q, out=out, off=off: m.paged_attention_forward(desc, q, off, kv, tab, *dev, out, workspace=ws))
              for _, _, q, out, off in calls]
    for _ in range(3):
        for graph, (q_lens, q, _, out, _) in zip(graphs, calls):
            out.fill_(float("nan"))
            graph.replay()
            want, tol, _ = paged64(q, _offsets(q_lens), lens, table, values, c)
            assert_within(out, want, tol)
    assert bool((ws[need:] == 255).all())


@pytest.mark.parametrize("batch", [4, 70])
@pytest.mark.parametrize("q_len", [1, 40])
def test_offsets_that_do_not_ascend(q_len, batch):
    """Offsets back and forth and beyond the rows: sequences whose offsets do not ascend have no rows, and nothing past
    out or the workspace is written."""
    m, ps, tokens = cc(), 16, 4 * q_len
    got, values = random_cache(60, ps, 2, 64, "bf16", "bf16", 5)
    dev = [got["k"].cuda(), got["v"].cuda(), None, None]
    lens = [200, 90, 300, 260] + [0] * (batch - 4)
    table = tables(lens, ps, 60, 20)
    q = torch.randn(tokens, 4, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    desc = _desc(4, 2, 64, ps, dict(dtype="bf16", cache="bf16"))
    guard = torch.full((tokens + 2, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    for offsets in ([2 * q_len, q_len, 3 * q_len, 0, -5], [tokens + 7, tokens, 3 * q_len, tokens + 100, 1]):
        offsets = offsets + [0] * (batch + 1 - len(offsets))
        guard.fill_(9.0)
        out = guard[1:tokens + 1]
        _run(desc, q.cuda(), offsets, lens, table.cuda(), dev, out=out)
        want, tol, mine = paged64(q, offsets, lens, table, values, dict(dtype="bf16", cache="bf16"))
        want[~mine], tol[~mine] = 9.0, 0.0
        assert_within(out, want, tol, str(offsets[:5]))
        assert bool((guard[0] == 9).all()) and bool((guard[-1] == 9).all())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_two_calls_at_once(cache):
    """Two streams with a workspace each, over the same pages."""
    m, ps, c = cc(), 16, dict(dtype="bf16", cache=cache)
    lens = [3000, 10, 1500]
    got, values = random_cache(300, ps, 2, 128, "bf16", cache, 7)
    dev = [None if got[n] is None else got[n].cuda() for n in ("k", "v", "ks", "vs")]
    table, desc = tables(lens, ps, 300, 200), _desc(8, 2, 128, ps, c)
    off, kv, tab = _ints([0, 1, 2, 3]), _ints(lens), table.cuda()
    n = m.paged_attention_workspace_bytes(desc, 3, 3, 200)
    sides = []
    for i in range(2):
        q = torch.randn(3, 8, 128, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16)
        sides.append((torch.cuda.Stream(), q, q.cuda(), torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda"),
                      torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, _, q, out, ws in sides:
            m.paged_attention_forward(desc, q, off, kv, tab, *dev, out, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for _, q, _, out, _ in sides:
        want, tol, _ = paged64(q, [0, 1, 2, 3], lens, table, values, c)
        assert_within(out, want, tol)


def test_wrong_tensors_are_refused():
    """Types, shapes, strides, other devices and workspaces, by the binding before anything runs."""
    m, ps = cc(), 16
    desc = _desc(4, 2, 64, ps, dict(dtype="bf16", cache="bf16"))
    t = dict(dtype=torch.bfloat16, device="cuda")
    q, out = torch.zeros(2, 4, 64, **t), torch.full((2, 4, 64), 9.0, **t)
    k, v = torch.zeros(200, ps, 2, 64, **t), torch.zeros(200, ps, 2, 64, **t)
    args = dict(q=q, off=_ints([0, 1, 2]), kv=_ints([3000, 9]), tab=torch.arange(400, dtype=torch.int32, device="cuda").view(2, 200) % 200,
                k=k, v=v, ks=None, vs=None, out=out)
    need = m.paged_attention_workspace_bytes(desc, 2, 2, 200)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def call(ws=ws, **kw):
        a = dict(args, **kw)
        m.paged_attention_forward(desc, a["q"], a["off"], a["kv"], a["tab"], a["k"], a["v"], a["ks"], a["vs"], a["out"], workspace=ws)
    for kw in (dict(q=q.cpu()), dict(q=q.float()), dict(q=q[:, :3]), dict(off=_ints([0, 1])), dict(kv=args["kv"].long()),
               dict(tab=args["tab"][:, ::2]), dict(k=k[:, :8]), dict(v=v.cpu()), dict(k=k.transpose(1, 2)), dict(out=out.float()),
               dict(kv=args["kv"].cpu()), dict(ws=ws.cpu()), dict(off=None), dict(out=None)):
        with pytest.raises((ValueError, TypeError, AttributeError, m.ConvError)):
            call(**kw)
    if need:
        for short in (None, ws[:-16]):
            with pytest.raises(m.ConvError):
                call(ws=short)
    torch.cuda.synchronize()
    assert bool((out == 9).all())
    call()
    assert bool((out == 0).all())
