"""GPU: keys, values and scales interleaved in one buffer: stored, read back and attended to."""
import pytest
import torch

from attention_reference import TYPES, assert_within
from decoder_reference import E4M3, paged64, quantise64

pytestmark = pytest.mark.gpu

HEADS, D, PS, PAGES = 4, 64, 8, 7


def _views(layout, dtype, cache):
    """(keys, values, scales of both) [page, token, head(, element)] in one buffer, and the buffer."""
    t = torch.uint8 if cache == "e4m3" else TYPES[dtype]
    new = lambda *s: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    scales = [None, None]
    if cache == "e4m3":
        scales = [torch.zeros(PAGES, PS, HEADS, dtype=torch.uint8, device="cuda") for _ in "kv"]
    if layout == "token":
        b = new(PAGES, PS, 2, HEADS, D)
        k, v = b[:, :, 0], b[:, :, 1]
    elif layout == "head":
        b = new(PAGES, PS, HEADS, 2, D)
        k, v = b[..., 0, :], b[..., 1, :]
    elif layout == "heads outermost":
        b = new(HEADS, 2, PAGES, PS, D)
        k, v = (b[:, i].permute(1, 2, 0, 3) for i in (0, 1))
    else:   # codes, their scale, 15 bytes that stay
        b = new(PAGES, PS, HEADS, 2, D + 16)
        k, v = b[..., 0, :D], b[..., 1, :D]
        scales = [b[..., i, D] for i in (0, 1)]
    return k, v, scales, b


@pytest.mark.parametrize("dtype,cache,layout", [(t, c, n) for t, c in (("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32"), ("f32", "e4m3"))
                                                for n in ("token", "head", "heads outermost", "scales") if n != "scales" or c == "e4m3"])
def test_interleaved(layout, dtype, cache):
    import convolution_conv2d_forward_amd as m
    t, g = TYPES[dtype], torch.Generator().manual_seed(5)
    k, v, scales, buffer = _views(layout, dtype, cache)
    strides = dict(k_page_strides=k.stride()[:3], v_page_strides=v.stride()[:3])
    if cache == "e4m3":
        strides["scale_strides"] = scales[0].stride()
        k, v = k.view(E4M3), v.view(E4M3)
    slots = torch.randperm(PAGES * PS, generator=g)
    x = torch.randn(2, PAGES * PS, HEADS, D, generator=g).to(t)
    ints = lambda a: torch.as_tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    desc = m.kv_cache_desc_create(m.make_kv_cache_params(HEADS, D, PS, dtype=dtype, cache_dtype=cache, **strides))
    m.kv_cache_store(desc, x[0].cuda(), x[1].cuda(), ints(slots), k, v, *scales)
    values = {}
    for n, rows in (("k", x[0]), ("v", x[1])):
        want = rows.double()
        if cache == "e4m3":
            codes, e = quantise64(rows)
            want = torch.ldexp(codes, e[..., None])
        values[n] = torch.zeros(PAGES * PS, HEADS, D, dtype=torch.float64).index_copy(0, slots, want).view(PAGES, PS, HEADS, D)
    if layout == "scales":
        assert (buffer[..., D + 1:] == 0).all()
    table, lens = torch.tensor([[3, 0, 6], [1, 5, 2]], dtype=torch.int32), [21, 17]
    wide = torch.full((2, 30, 2, HEADS, D), 5.0, dtype=t, device="cuda")
    out = wide[:, :24]
    s = dict(k_stride=2 * HEADS * D, v_stride=2 * HEADS * D, k_batch_stride=wide.stride(0), v_batch_stride=wide.stride(0))
    load = m.kv_cache_desc_create(m.make_kv_cache_params(HEADS, D, PS, dtype=dtype, cache_dtype=cache, **strides, **s))
    m.kv_cache_load(load, ints(table), ints(lens), k, v, *scales, out[:, :, 0], out[:, :, 1])
    for i, n in enumerate("kv"):
        for b, length in enumerate(lens):
            want = values[n][table[b].long()].flatten(0, 1)[:length]
            assert torch.equal(out[b, :length, i].cpu().double(), want)
            assert (wide[b, length:, i] == 5).all()
    q = torch.randn(3, 8, D, generator=g).to(t)
    att = m.paged_attention_desc_create(m.make_paged_attention_params(8, HEADS, D, PS, dtype=dtype, cache_dtype=cache, **strides))
    n = m.paged_attention_workspace_bytes(att, 3, 2, 3)
    got = torch.zeros_like(q, device="cuda")
    m.paged_attention_forward(att, q.cuda(), ints([0, 2, 3]), ints(lens), ints(table), k, v, *scales, got,
                              workspace=torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None)
    want, tol, _ = paged64(q, [0, 2, 3], lens, table, values, dict(dtype=dtype))
    assert_within(got, want, tol)
