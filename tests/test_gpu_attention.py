"""GPU: attention_forward against the 64-bit definition: every mask and bias,
single tokens to prompts, grouped heads, ragged lengths, rows that see nothing,
garbage in places that no row sees."""
import pytest
import torch

from attention_reference import TYPES, assert_within, attention64

pytestmark = pytest.mark.gpu


def cc():
    import convolution_conv2d_forward_amd as m
    return m


def _ints(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


def _inputs(b, q_len, kv_len, hq, hk, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    return ((2 * torch.randn(b, q_len, hq, d, generator=g)).to(t), torch.randn(b, kv_len, hk, d, generator=g).to(t),
            torch.randn(b, kv_len, hk, d, generator=g).to(t))


def _call(q, k, v, c, out=None, q_lens=None, kv_lens=None, prefix=None, docs=None, slopes=None):
    """Device tensors; returns out, filled with NaN before."""
    if out is None:
        out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    d = cc().attention_desc_create(cc().make_attention_params(
        q.shape[2], k.shape[2], q.shape[3], q_strides=q.stride()[:3], k_strides=k.stride()[:3],
        v_strides=v.stride()[:3], out_strides=out.stride()[:3], causal=c.get("causal", False),
        window=c.get("window", 0), softcap=c.get("softcap", 0.0), scale=c.get("scale"), has_slopes=slopes is not None,
        dtype=c["dtype"]))
    n = cc().attention_workspace_bytes(d, q.shape[0], q.shape[1], k.shape[1])
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None
    cc().attention_forward(d, q, k, v, out, q_lens=_ints(q_lens), kv_lens=_ints(kv_lens), prefix_lens=_ints(prefix),
                           doc_offsets=_ints(docs), slopes=None if slopes is None else slopes.cuda(), workspace=ws)
    return out


def _check(b, q_len, kv_len, hq, hk, d, dtype, seed=0, slopes=False, **kw):
    c = {n: kw[n] for n in ("causal", "window", "softcap", "scale") if n in kw}
    c["dtype"] = dtype
    lens = {n: kw[n] for n in ("q_lens", "kv_lens", "prefix", "docs") if n in kw}
    q, k, v = _inputs(b, q_len, kv_len, hq, hk, d, dtype, seed)
    if slopes:
        lens["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1) / hq).float()
    got = _call(q.cuda(), k.cuda(), v.cuda(), c, **lens)
    want, tol = attention64(q, k, v, c, lens.get("q_lens"), lens.get("kv_lens"), lens.get("prefix"), lens.get("docs"),
                            lens.get("slopes"))
    assert_within(got, want, tol, f"{b} {q_len}/{kv_len} {hq}/{hk} d{d} {dtype} {kw}")


DIMS = {"f32": [4, 20, 32, 64, 96, 100, 128, 160, 256], "bf16": [8, 24, 32, 64, 80, 96, 128, 136, 192, 256]}


@pytest.mark.parametrize("dtype,d", [(t, d) for t, ds in DIMS.items() for d in ds])
@pytest.mark.parametrize("q_len", [1, 70])
def test_head_dims(dtype, d, q_len):
    _check(2, q_len, 150, 4, 2, d, dtype, causal=True, softcap=30.0)


LENGTHS = [(1, 1), (1, 2), (1, 31), (1, 33), (1, 64), (1, 257), (1, 1100), (2, 2), (3, 500), (5, 17), (8, 1030), (16, 16),
           (17, 900), (33, 70), (64, 64), (65, 130), (127, 127), (129, 129), (200, 333), (256, 300), (300, 300), (7, 3)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("q_len,kv_len", LENGTHS)
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(q_len, kv_len, causal, dtype):
    """(7, 3): the first rows of a causal block are before every key."""
    _check(1, q_len, kv_len, 4, 1, 64, dtype, causal=causal)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (6, 2), (5, 1), (16, 1), (32, 4), (24, 1)])
@pytest.mark.parametrize("q_len", [1, 4, 50])
def test_groups(hq, hk, q_len, dtype):
    _check(2, q_len, 90, hq, hk, 128, dtype, causal=True, slopes=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("q_len,kv_len", [(1, 400), (6, 300), (180, 180), (140, 400)])
@pytest.mark.parametrize("kw", [
    dict(softcap=20.0), dict(slopes=True), dict(softcap=8.0, slopes=True, causal=True), dict(window=1, causal=True),
    dict(window=40, causal=True), dict(window=65), dict(window=2 ** 31 - 1, causal=True), dict(scale=0.5, causal=True),
    dict(prefix=[0, 33], causal=True), dict(prefix=[1000, -5], causal=True), dict(prefix=[64, 100], causal=True, window=50),
    dict(docs=[[0, 1, 1, 64, 100, 180], [0, 0, 50, 51, 170, 400]], causal=True),
    dict(docs=[[0, 90, 90, 90, 91, 120], [10, 20, 60, 64, 128, 150]]),
    dict(docs=[[0, 180, 400], [0, 32, 400]], slopes=True, softcap=50.0),
], ids=lambda kw: "-".join(kw))
def test_masks_and_biases(kw, q_len, kv_len, dtype):
    _check(2, q_len, kv_len, 4, 2, 64, dtype, **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("q_len,kv_len", [(1, 700), (4, 700), (150, 150), (100, 300)])
@pytest.mark.parametrize("causal", [False, True])
def test_ragged_lengths(q_len, kv_len, causal, dtype):
    """Empty sequences, single keys, lengths beyond the buffers (clamped),
    fewer keys than queries; rows past a sequence's end are zero."""
    kv = [kv_len, 0, 1, kv_len + 99, 33, min(2, kv_len)]
    ql = [q_len, q_len, 1, q_len // 2, -4, q_len]
    _check(6, q_len, kv_len, 4, 2, 64, dtype, q_lens=ql, kv_lens=kv, causal=causal)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("q_len,kv_len", [(1, 200), (3, 600), (150, 150), (90, 280)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_unseen_garbage_does_not_spread(bad, q_len, kv_len, dtype):
    """Infinities and NaN past a sequence's length, in the future of causal
    rows, in other documents and outside the window."""
    c = {"dtype": dtype, "causal": True, "window": 60}
    docs = [[0, 40, 100, kv_len]] * 2
    q, k, v = _inputs(2, q_len, kv_len, 4, 2, 64, dtype, 4)
    lens = [kv_len, kv_len - 25]
    k[1, lens[1]:] = bad
    v[1, lens[1]:] = bad
    v[0, kv_len - 1, 0, 3] = bad      # the last key: seen by the last row alone
    v[0, 45, 1, 7] = bad
    k[0, 20] = bad if bad != bad else 0.0
    got = _call(q.cuda(), k.cuda(), v.cuda(), c, kv_lens=lens, docs=docs)
    want, tol = attention64(q, k, v, c, None, lens, None, docs)
    # A NaN key makes the rows that see it NaN, whole; the reference says where.
    assert_within(got, want, tol, f"{bad}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_scores(dtype):
    """Scores of thousands: weights of 0 and 1, no overflow; and scores all
    equal to a large negative number."""
    q, k, v = _inputs(1, 40, 200, 2, 1, 64, dtype, 6)
    for f in (300.0, -300.0):
        qf = (q * f).to(q.dtype)
        c = {"dtype": dtype, "causal": True}
        got = _call(qf.cuda(), k.cuda(), v.cuda(), c).cpu().double()
        assert torch.isfinite(got).all()
        assert (got.abs() <= v.double().abs().max() * (1 + 2.0 ** -7)).all()
    one = torch.ones_like(q) * -30.0
    k1 = torch.ones_like(k) * 30.0
    got = _call(one.cuda(), k1.cuda(), v.cuda(), {"dtype": dtype})
    want, tol = attention64(one, k1, v, {"dtype": dtype})
    assert_within(got, want, tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("q_len", [1, 80])
def test_layouts(q_len, dtype):
    """q, k and v inside one projection buffer; the cache as [head][token]; out
    as [head][token]; a key repeated over the batch by stride 0."""
    b, L, hq, hk, d = 2, 80, 6, 3, 64
    t, c = TYPES[dtype], {"dtype": dtype, "causal": True}
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(b, L, (hq + 2 * hk) * d, generator=g).to(t)
    parts = [x.unflatten(-1, (-1, d)) for x in qkv.cuda().split([hq * d, hk * d, hk * d], -1)]
    host = [x.unflatten(-1, (-1, d)) for x in qkv.split([hq * d, hk * d, hk * d], -1)]
    want, tol = attention64(host[0][:, L - q_len:], host[1], host[2], c)
    q = parts[0][:, L - q_len:]
    assert_within(_call(q, parts[1], parts[2], c, out=torch.empty(q.shape, dtype=t, device="cuda")), want, tol)
    k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in parts[1:])
    out = torch.empty((b, hq, q_len, d), dtype=t, device="cuda").transpose(1, 2)
    assert_within(_call(q, k, v, c, out=out), want, tol)
    k1, v1 = (x[:1].expand(b, -1, -1, -1) for x in (k, v))
    want, tol = attention64(host[0][:, L - q_len:], host[1][:1].expand(b, -1, -1, -1), host[2][:1].expand(b, -1, -1, -1), c)
    assert_within(_call(q, k1, v1, c, out=out), want, tol)


@pytest.mark.parametrize("q_len", [1, 70])
def test_cache_beyond_32_bit_offsets(q_len):
    hk, d, L, stride = 2, 64, 300, 1 << 24
    q, k, v = _inputs(1, q_len, L, 4, hk, d, "bf16", 8)
    buf = torch.empty((L - 1) * stride + 2 * hk * d, dtype=torch.bfloat16, device="cuda")
    kc = buf.as_strided((1, L, hk, d), (0, stride, d, 1))
    vc = buf.as_strided((1, L, hk, d), (0, stride, d, 1), hk * d)
    kc.copy_(k)
    vc.copy_(v)
    c = {"dtype": "bf16", "causal": True}
    want, tol = attention64(q, k, v, c)
    assert_within(_call(q.cuda(), kc, vc, c), want, tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_cache_and_same_results_twice(dtype):
    q, k, v = _inputs(2, 1, 9000, 8, 2, 128, dtype, 11)
    lens = [9000, 4097]
    slopes = torch.exp2(-torch.arange(1, 9).float())
    c = {"dtype": dtype, "causal": True, "softcap": 50.0}
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    got = _call(qd, kd, vd, c, kv_lens=lens, slopes=slopes)
    want, tol = attention64(q, k, v, c, None, lens, None, None, slopes)
    assert_within(got, want, tol)
    assert torch.equal(got, _call(qd, kd, vd, c, kv_lens=lens, slopes=slopes))


def test_no_keys_and_no_queries():
    q, k, v = (x.cuda() for x in _inputs(2, 5, 1, 4, 2, 64, "bf16"))
    c = {"dtype": "bf16"}
    assert (_call(q, k[:, :0], v[:, :0], c) == 0).all()
    assert _call(q[:, :0], k, v, c).numel() == 0
    assert _call(q[:0], k[:0], v[:0], c).numel() == 0


def test_bad_document_offsets_stay_inside_the_sequence():
    """Offsets that do not ascend or point past the cache read nothing outside
    it; which keys are seen is not defined."""
    q, k, v = (x.cuda() for x in _inputs(1, 60, 60, 2, 1, 64, "bf16"))
    for docs in ([[50, 3, 900, -7, 60]], [[2 ** 30, 2 ** 31 - 1, 0, 5, 5]], [[-5, 2 ** 31 - 1, 2 ** 31 - 1, 0, 0]]):
        got = _call(q, k, v, {"dtype": "bf16"}, docs=docs)
        assert torch.isfinite(got).all()


@pytest.mark.parametrize("q_len", [1, 70])
def test_graph_replays_and_streams(q_len):
    """rope, attention and linear captured together; every replay, with eager
    work between, gives what the eager calls give on the values of that time."""
    m, hq, hk, d, L = cc(), 4, 2, 64, 1500
    t = torch.bfloat16
    width = (hq + 2 * hk) * d
    qkv = torch.randn(q_len, width, device="cuda").to(t)
    pos = torch.arange(L - q_len, L, dtype=torch.int32, device="cuda")
    slots = pos.clone()
    kc, vc = (torch.randn(L, hk, d, device="cuda").to(t) for _ in "kv")
    w = (torch.randn(hq * d, hq * d, device="cuda") / 16).to(t)
    q, o = (torch.empty(q_len, hq, d, dtype=t, device="cuda") for _ in "qo")
    y = torch.zeros(q_len, hq * d, dtype=t, device="cuda")
    rope = m.qk_rope_desc_create(m.make_qk_rope_params(hq, hk, d, dtype="bf16"))
    q4, k4, v4, o4 = (x.unsqueeze(0) for x in (q, kc, vc, o))
    att = m.attention_desc_create(m.make_attention_params(
        hq, hk, d, q_strides=q4.stride()[:3], k_strides=k4.stride()[:3], v_strides=v4.stride()[:3],
        out_strides=o4.stride()[:3], causal=True, dtype="bf16"))
    lin = m.linear_desc_create(m.make_linear_params(hq * d, hq * d, has_residual=True, dtype="bf16"))
    ws = torch.empty(max(1, m.attention_workspace_bytes(att, 1, q_len, L)), dtype=torch.uint8, device="cuda")
    res = torch.randn(q_len, hq * d, device="cuda").to(t)

    def layer():
        m.qk_rope_forward(rope, qkv, None, None, pos, slots, q, kc, vc)
        m.attention_forward(att, q4, k4, v4, o4, workspace=ws)
        m.linear_forward(lin, o.view(q_len, hq * d), w, None, res, y)

    layer()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for i in range(4):
        qkv.copy_(torch.randn(q_len, width, device="cuda").to(t))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        y.zero_()
        layer()
        torch.cuda.synchronize()
        assert torch.equal(got, y), i
