"""GPU: qk_rope_forward against the 64-bit definition: layouts, partial heads,
scalings, far positions, cache slots, strides, odd head sizes, in place."""
import pytest
import torch

from attention_reference import TYPES, assert_within, rope64

pytestmark = pytest.mark.gpu


def cc():
    import convolution_conv2d_forward_amd as m
    return m


def _case(**kw):
    c = dict(tokens=9, heads_q=4, heads_kv=2, head_dim=64, rotary_dim=64, layout="half", has_norm=True, eps=1e-6,
             theta=10000.0, scaling="none", factor=1.0, original_len=0, dtype="bf16", last=500)
    c.update(kw)
    return c


def _desc(c, **strides):
    names = ("rotary_dim", "layout", "has_norm", "eps", "theta", "scaling", "factor", "original_len", "dtype")
    return cc().qk_rope_desc_create(cc().make_qk_rope_params(
        c["heads_q"], c["heads_kv"], c["head_dim"], **{n: c[n] for n in names}, **strides))


def _inputs(c, seed=0):
    g = torch.Generator().manual_seed(seed)
    t, hq, hk, d = c["tokens"], c["heads_q"], c["heads_kv"], c["head_dim"]
    qkv = (3 * torch.randn(t, (hq + 2 * hk) * d, generator=g)).to(TYPES[c["dtype"]])
    gq, gk = (1 + 0.3 * torch.randn(d, generator=g) for _ in "qk")
    pos = torch.randint(-3, c["last"] + 1, (t,), generator=g, dtype=torch.int32)
    pos[0] = c["last"]
    return qkv, gq, gk, pos


def _want(c, qkv, gq, gk, pos):
    t, hq, hk, d = c["tokens"], c["heads_q"], c["heads_kv"], c["head_dim"]
    x = qkv.view(t, hq + 2 * hk, d)
    n = c["has_norm"]
    return (rope64(x[:, :hq], gq if n else None, pos, c), rope64(x[:, hq:hq + hk], gk if n else None, pos, c),
            x[:, hq + hk:])


def _check(c, seed=0):
    qkv, gq, gk, pos = _inputs(c, seed)
    t, hq, hk, d = c["tokens"], c["heads_q"], c["heads_kv"], c["head_dim"]
    (q, tq), (k, tk), v = _want(c, qkv, gq, gk, pos)
    dt = TYPES[c["dtype"]]
    out = [torch.full((t, h, d), float("nan"), dtype=dt, device="cuda") for h in (hq, hk, hk)]
    cc().qk_rope_forward(_desc(c), qkv.cuda(), gq.cuda(), gk.cuda(), pos.cuda(), None, *out)
    assert_within(out[0], q, tq, f"q {c}")
    assert_within(out[1], k, tk, f"k {c}")
    assert torch.equal(out[2].cpu(), v), "values are copied"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("head_dim,rotary", [(8, 8), (32, 16), (64, 64), (80, 40), (96, 24), (128, 128), (128, 32),
                                             (256, 256), (256, 128), (2, 2), (5, 4), (63, 10), (100, 100), (200, 6)])
def test_heads(head_dim, rotary, layout, dtype):
    _check(_case(head_dim=head_dim, rotary_dim=rotary, layout=layout, dtype=dtype))


@pytest.mark.parametrize("heads_q,heads_kv,tokens", [(1, 1, 1), (7, 1, 1), (32, 8, 1), (6, 6, 37), (16, 2, 400),
                                                     (3, 1, 2500)])
@pytest.mark.parametrize("norm", [False, True])
def test_counts(heads_q, heads_kv, tokens, norm):
    _check(_case(heads_q=heads_q, heads_kv=heads_kv, tokens=tokens, has_norm=norm))


@pytest.mark.parametrize("scaling,factor,original", [("none", 1.0, 0), ("linear", 8.0, 0), ("yarn", 4.0, 2048),
                                                     ("yarn", 32.0, 64), ("yarn", 1.0, 4096)])
@pytest.mark.parametrize("last", [1, 131071, 2 ** 31 - 1])
def test_scaled_and_far_positions(scaling, factor, original, last):
    """The last position: an fp32 angle there would be wrong by whole turns."""
    _check(_case(scaling=scaling, factor=factor, original_len=original, last=last, dtype="f32", theta=500000.0))


@pytest.mark.parametrize("vec", [True, False])
def test_slots_store_only_their_rows(vec):
    c = _case(tokens=6, head_dim=64 if vec else 60, rotary_dim=64 if vec else 60)
    qkv, gq, gk, pos = _inputs(c)
    (q, tq), (k, tk), v = _want(c, qkv, gq, gk, pos)
    slots = torch.tensor([7, 0, -1, 11, 12, 3], dtype=torch.int32)   # -1 and 12 lie outside the cache
    kc, vc = (torch.full((12, 2, c["head_dim"]), 5.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    qo = torch.empty((6, 4, c["head_dim"]), dtype=torch.bfloat16, device="cuda")
    cc().qk_rope_forward(_desc(c), qkv.cuda(), gq.cuda(), gk.cuda(), pos.cuda(), slots.cuda(), qo, kc, vc)
    assert_within(qo, q, tq)
    kept = [0, 1, 3, 5]
    rows = slots[kept].long()
    assert_within(kc[rows.cuda()], k[kept], tk[kept])
    assert torch.equal(vc.cpu()[rows], v[kept])
    others = [r for r in range(12) if r not in rows.tolist()]
    assert (kc[others] == 5).all() and (vc[others] == 5).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift,pad", [(0, 16), (8, 8), (1, 3)])
def test_strided_in_place_and_without_values(shift, pad, dtype):
    """Queries in place inside a wider qkv buffer, keys to strided rows, values
    not stored; aligned and unaligned."""
    c = _case(dtype=dtype, tokens=11)
    qkv, gq, gk, pos = _inputs(c)
    (q, tq), (k, tk), _ = _want(c, qkv, gq, gk, pos)
    t, width, dt = 11, qkv.shape[1], TYPES[dtype]
    wide = torch.full((t, width + 32 + pad), 3.0, dtype=dt, device="cuda")
    s = width + 32 + pad
    inner = wide[:, shift:shift + width]
    inner.copy_(qkv)
    qv = wide.as_strided((t, 4, 64), (s, 64, 1), shift)
    kbuf = torch.full((t, 128 + pad), 9.0, dtype=dt, device="cuda")
    kv = kbuf.as_strided((t, 2, 64), (128 + pad, 64, 1))
    d = _desc(c, qkv_stride=s, q_stride=s, k_stride=128 + pad)
    cc().qk_rope_forward(d, inner, gq.cuda(), gk.cuda(), pos.cuda(), None, qv, kv, None)
    assert_within(qv, q, tq)
    assert_within(kv, k, tk)
    assert torch.equal(inner[:, 256:].cpu(), qkv[:, 256:]) and (kbuf[:, 128:] == 9).all()


def test_cache_rows_beyond_32_bit_offsets():
    c = _case(tokens=3, heads_kv=1, heads_q=1)
    qkv, gq, gk, pos = _inputs(c)
    (q, tq), (k, tk), v = _want(c, qkv, gq, gk, pos)
    stride, rows = 1 << 20, 4500
    kbuf = torch.empty((rows - 1) * stride + 64, dtype=torch.bfloat16, device="cuda")
    kc = kbuf.as_strided((rows, 1, 64), (stride, 64, 1))
    vc = torch.empty((rows, 1, 64), dtype=torch.bfloat16, device="cuda")
    qo = torch.empty((3, 1, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([4499, 0, 2200], dtype=torch.int32)
    cc().qk_rope_forward(_desc(c, k_stride=stride), qkv.cuda(), gq.cuda(), gk.cuda(), pos.cuda(), slots.cuda(), qo, kc,
                         vc)
    assert_within(kc[slots.long().cuda()], k, tk)
    assert torch.equal(vc.cpu()[slots.long()], v)
