"""GPU: the attention-layer kernels at sizes that choose each of them, their rules' borders, and the example layer."""
import os
import sys

import pytest
import torch

from attention_reference import TYPES, assert_within, attention64, linear64

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def cc():
    import convolution_conv2d_forward_amd as m
    return m


# -------------------------------------------------------------- linear --

@pytest.mark.parametrize("m,k,n,dtype,kernel", [
    (1, 200, 64, "bf16", "linear_rows_bf16"), (16, 72, 50, "f32", "linear_rows_f32"),
    (17, 136, 100, "bf16", "linear_rows_bf16"), (40, 2056, 200, "bf16", "linear_rows_bf16"),
    (64, 72, 1000, "f32", "linear_rows_f32"), (65, 264, 130, "bf16", "linear_rows_bf16"),
    (128, 520, 48, "bf16", "linear_rows_bf16"), (100, 100, 33, "f32", "linear_rows_f32"),
    (200, 328, 264, "bf16", "linear_rows_bf16"), (129, 36, 100, "f32", "linear_rows_f32"),
    (46, 264, 100, "f32", "linear_rows_f32"), (100, 136, 600, "f32", "linear_rows_f32"),
    (100, 134, 600, "bf16", "linear_rows_bf16"), (100, 133, 600, "f32", "linear_rows_f32"),
    (40, 2056, 4100, "bf16", "linear_rows_bf16"), (40, 1029, 4100, "f32", "linear_rows_f32"),
    (40, 333, 100, "bf16", "linear_rows_bf16"),
    (1000, 72, 1000, "bf16", "linear_tile_bf16/64"), (1000, 32, 1000, "f32", "linear_tile_f32/64"),
    (1000, 136, 4000, "bf16", "linear_tile_bf16/128deep"), (2000, 44, 2000, "f32", "linear_tile_f32/128deep"),
    (2000, 72, 4000, "bf16", "linear_tile_bf16/128"), (4090, 72, 4088, "bf16", "linear_tile_bf16/256"),
    (4096, 8, 4090, "bf16", "linear_tile_bf16/256"),
    # Rows at 4-byte boundaries, and at none.
    (300, 66, 257, "bf16", "linear_tile_bf16/64"), (2000, 70, 3001, "bf16", "linear_tile_bf16/128"),
    (300, 37, 65, "f32", "linear_tile_f32/64"), (1990, 33, 2001, "f32", "linear_tile_f32/128deep"),
    (300, 67, 130, "bf16", "linear_tile_bf16/64"), (70, 515, 100, "bf16", "linear_rows_bf16"),
    (70, 514, 100, "bf16", "linear_rows_bf16"), (33, 515, 49, "f32", "linear_rows_f32"),
    (2000, 35, 3001, "bf16", "linear_tile_bf16/128"),
    (50, 33, 40, "bf16", "linear_tile_bf16/64"),
])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_linear_kernels(m, k, n, dtype, kernel, act):
    g = torch.Generator().manual_seed(m + k + n)
    t = TYPES[dtype]
    x, w = torch.randn(m, k, generator=g).to(t), (torch.randn(n, k, generator=g) * k ** -0.5).to(t)
    b, r = torch.randn(n, generator=g), torch.randn(m, n, generator=g).to(t)
    d = cc().linear_desc_create(cc().make_linear_params(k, n, has_bias=True, has_residual=True, act=act, dtype=dtype))
    if k * x.element_size() % 16 == 0:   # the name is for rows at 16-byte boundaries
        assert cc().linear_desc_kernel_name(d, m) == kernel
    guard = torch.full((m + 2, n), 7.0, dtype=t, device="cuda")
    y = guard[1:m + 1]
    cc().linear_forward(d, x.cuda(), w.cuda(), b.cuda(), r.cuda(), y)
    want, tol = linear64(x, w, b, r, dtype, act)
    assert_within(y, want, tol, f"{m}x{k}x{n} {dtype}")
    assert (guard[0] == 7).all() and (guard[-1] == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [20, 90, 700])
def test_linear_reads_nothing_past_its_rows(m, dtype):
    """NaN beside the rows of x and behind w: chunks past k are zero, whatever lies there."""
    k, n, t = 72, 80, TYPES[dtype]
    g = torch.Generator().manual_seed(4)
    x, w = torch.randn(m, k, generator=g).to(t), torch.randn(n, k, generator=g).to(t)
    wide = torch.full((m + 1, k + 8), float("nan"), dtype=t, device="cuda")
    behind = torch.full((n + 1, k), float("nan"), dtype=t, device="cuda")
    wide[:m, :k], behind[:n] = x, w
    d = cc().linear_desc_create(cc().make_linear_params(k, n, x_stride=k + 8, dtype=dtype))
    y = torch.empty((m, n), dtype=t, device="cuda")
    cc().linear_forward(d, wide[:m, :k], behind[:n], None, None, y)
    want, tol = linear64(x, w, None, None, dtype)
    assert_within(y, want, tol)


# ----------------------------------------------------------- attention --

def _ints(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


def _check(b, q_len, kv_len, hq, hk, d, dtype, seed=0, slopes=False, kv_lens=None, q_lens=None, docs=None, prefix=None,
           spoil=None, **c):
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    q = (2 * torch.randn(b, q_len, hq, d, generator=g)).to(t)
    k, v = (torch.randn(b, kv_len, hk, d, generator=g).to(t) for _ in "kv")
    if spoil:
        spoil(k, v)
    s = torch.exp2(-8.0 * torch.arange(1, hq + 1) / hq).float() if slopes else None
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    out = torch.full(q.shape, float("nan"), dtype=t, device="cuda")
    m = cc()
    desc = m.attention_desc_create(m.make_attention_params(
        hq, hk, d, q_strides=qd.stride()[:3], k_strides=kd.stride()[:3], v_strides=vd.stride()[:3],
        out_strides=out.stride()[:3], has_slopes=slopes, dtype=dtype, **c))
    n = m.attention_workspace_bytes(desc, b, q_len, kv_len)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None
    m.attention_forward(desc, qd, kd, vd, out, q_lens=_ints(q_lens), kv_lens=_ints(kv_lens), prefix_lens=_ints(prefix),
                        doc_offsets=_ints(docs), slopes=None if s is None else s.cuda(), workspace=ws)
    want, tol = attention64(q, k, v, dict(c, dtype=dtype), q_lens, kv_lens, prefix, docs, s)
    assert_within(out, want, tol)
    return n


@pytest.mark.parametrize("dtype,d,c", [
    ("bf16", 64, dict(causal=True, softcap=30.0)), ("bf16", 32, dict(window=100)), ("f32", 32, dict(causal=True)),
    ("bf16", 128, dict(causal=True, slopes=True)), ("f32", 40, dict(causal=True, softcap=20.0, slopes=True)),
])
def test_enough_rows_for_whole_tiles(dtype, d, c):
    """512 tiles of 128 rows and more: neither the rows nor the keys are divided."""
    assert _check(2, 210, 210, 256, 128, d, dtype, kv_lens=[210, 77], q_lens=[210, 77], **c) == 0


@pytest.mark.parametrize("d,batch,kv_len,c", [
    (256, 2, 140, dict(causal=True)), (200, 2, 333, dict(softcap=30.0, slopes=True)), (256, 1, 1100, dict(window=300)),
])
def test_wide_heads(d, batch, kv_len, c):
    """Heads beyond 128 in 128-row tiles, from 192 of them on, and in 64-row tiles below; long keys are divided."""
    for heads in (50, 47):
        _check(batch, 140 if batch == 2 else 500, kv_len, heads, heads, d, "bf16",
               kv_lens=None if batch == 1 else [kv_len, kv_len - 131], **c)


def test_unseen_garbage_in_whole_tiles():
    def spoil(k, v):
        v[0, 205, 3, 5] = float("inf")     # seen by the last rows alone
        v[1, 60:, 7] = float("nan")        # past the second sequence
        v[0, 100, 9, 31] = float("nan")
    assert _check(2, 210, 210, 256, 128, 32, "bf16", kv_lens=[210, 60], q_lens=[210, 60], causal=True, spoil=spoil) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch", [40, 70])
def test_many_ragged_sequences(batch, dtype):
    """The workgroups' order goes by length for up to 64 sequences."""
    lens = [(37 * i) % 300 for i in range(batch)]
    _check(batch, 1, 300, 4, 2, 64, dtype, kv_lens=lens, causal=True)


@pytest.mark.parametrize("q_len", [1, 20, 150])
def test_many_documents(q_len):
    docs = [sorted((i * 7) % 301 for i in range(80)) + [300]]
    docs[0].sort()
    _check(1, q_len, 300, 4, 2, 64, "bf16", docs=docs, causal=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("q_len", [1, 6, 90])
def test_negative_scale(q_len, dtype):
    _check(1, q_len, 200, 4, 2, 64, dtype, scale=-0.2, softcap=10.0)
    _check(1, q_len, 200, 4, 2, 64, dtype, scale=-0.2, causal=True)


def test_more_splits_than_a_join_keeps_in_flight():
    assert _check(1, 2, 20011, 2, 1, 128, "bf16", causal=True) > 0
    assert _check(1, 1, 9001, 3, 1, 256, "f32", softcap=30.0) > 0


# ---------------------------------------------------------- the example --

@pytest.mark.parametrize("dtype,tol", [("bf16", 2.0 ** -5), ("f32", 2.0 ** -15)])
def test_example_layer_steps_match_its_prompt(dtype, tol):
    """The same tokens through other kernels.  An output of size 10 passes some ten roundings on its way: 10 * 2^-8
    for bf16 where all add up; fp32 sums of a few thousand terms stay below 2^-15 of it."""
    import attention_layer
    want, got, _, _ = attention_layer.run(tokens=300, steps=5, width=256, heads_q=4, heads_kv=2, head_dim=64,
                                          hidden=512, dtype=dtype)
    assert torch.isfinite(got).all()
    size = float(want.abs().max())
    assert float((got.double() - want.double()).abs().max()) <= tol * size
