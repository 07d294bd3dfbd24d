"""GPU: block_norm_forward against its 64-bit definition: norms, gates and scales, widths that choose each kernel, odd
widths, strides, the forms in place, rows of zeros and of one value."""
import pytest
import torch

from attention_reference import TYPES, assert_within
from decoder_reference import block_norm64

pytestmark = pytest.mark.gpu


def cc():
    import convolution_conv2d_forward_amd as m
    return m


def _inputs(rows, width, c, betas, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = TYPES[c["dtype"]]
    y, x = (2 * torch.randn(rows, width, generator=g) + 0.5).to(t), torch.randn(rows, width, generator=g).to(t)
    gate = None
    if c["gate_rows"] is not None:
        gate = torch.randn(-(-rows // c["gate_rows"]) if c["gate_rows"] else 1, width, generator=g).to(t)
    v = []
    for kind in (c["post"], c["pre"]):
        v.append(1 + 0.2 * torch.randn(width, generator=g) if kind != "none" else None)
        v.append(torch.randn(width, generator=g) if kind != "none" and betas else None)
    return y, x, gate, v


def _call(c, y, x, gate, v, residual, out, **strides):
    m = cc()
    d = m.block_norm_desc_create(m.make_block_norm_params(
        y.shape[1], post_norm=c["post"], pre_norm=c["pre"], has_post_beta=v[1] is not None,
        has_pre_beta=v[3] is not None, has_gate=gate is not None, gate_rows=c["gate_rows"] or 0,
        residual_scale=c["residual_scale"], block_scale=c["block_scale"], eps=c["eps"], dtype=c["dtype"], **strides))
    m.block_norm_forward(d, y, x, gate, *(None if t is None else t.cuda() for t in v), residual, out)


def _case(dtype, post="rms", pre="rms", gate_rows=None, residual_scale=1.0, block_scale=1.0, eps=1e-6):
    return dict(dtype=dtype, post=post, pre=pre, gate_rows=gate_rows, residual_scale=residual_scale,
                block_scale=block_scale, eps=eps)


def _check(rows, width, c, betas=False, seed=0, change=None):
    y, x, gate, v = _inputs(rows, width, c, betas, seed)
    if change:
        change(y, x)
    guard = [torch.full((rows + 2, width), 9.0, dtype=y.dtype, device="cuda") for _ in "ro"]
    r, o = guard[0][1:-1], guard[1][1:-1]
    _call(c, y.cuda(), x.cuda(), None if gate is None else gate.cuda(), v, r, o if c["pre"] != "none" else None)
    (wr, tr), rest = block_norm64(y, x, gate, v, c)
    assert_within(r, wr, tr, "residual")
    if rest:
        assert_within(o, *rest, "out")
    for t in guard:
        assert (t[0] == 9).all() and (t[-1] == 9).all()


WIDTHS = [1, 2, 7, 8, 63, 64, 72, 500, 512, 520, 1000, 1023, 1024, 1032, 2047, 2048, 2056, 4095, 4096, 4104, 8192, 8200,
          8201, 16384, 16392, 20001, 32767, 32768]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(width, dtype):
    _check(3, width, _case(dtype, "layer" if width > 1 else "rms", "rms", 0, 0.5, 2.0), betas=True, seed=width)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [40, 300, 2304])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("gate_rows", [None, 0, 1, 5])
def test_forms(gate_rows, pre, post, width, dtype):
    _check(13, width, _case(dtype, post, pre, gate_rows, 0.7, -1.3), betas=gate_rows == 5, seed=width)


@pytest.mark.parametrize("rows", [0, 1, 1000, 20000, 70001])
def test_rows(rows):
    """More rows than workgroups."""
    if rows == 0:
        t = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
        return _call(_case("bf16"), t, t, None, [torch.ones(64), None, torch.ones(64), None], t.clone(), t.clone())
    _check(rows, 64, _case("bf16", "none", "rms", 3), seed=rows)
    _check(rows, 40, _case("f32", "layer", "none"), seed=rows)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [64, 65, 4096])
def test_rows_without_spread(width, dtype):
    """Zeros, one value (its variance is rounding alone), a row far from zero, tiny and large numbers."""
    def change(y, x):
        y[0], x[0] = 0, 0
        y[1], x[1] = 3.0, -3.0
        y[2] += 1000
        y[3] *= 1e-6
        y[4] *= 1e15
    _check(6, width, _case(dtype, "rms", "rms"), change=change)
    _check(6, width, _case(dtype, "layer", "rms", eps=1e-3), change=change)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_numbers_stay_in_their_row(bad):
    c = _case("bf16")
    y, x, _, v = _inputs(9, 2048, c, False)
    y[4, 77] = bad
    r, o = torch.empty_like(y, device="cuda"), torch.empty_like(y, device="cuda")
    _call(c, y.cuda(), x.cuda(), None, v, r, o)
    keep = torch.arange(9) != 4
    (wr, tr), (wo, to) = block_norm64(y[keep], x[keep], None, v, c)
    assert_within(r.cpu()[keep], wr, tr)
    assert_within(o.cpu()[keep], wo, to)
    assert not torch.isfinite(o[4].float()).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [96, 97, 3001])
def test_in_place(width, dtype):
    """The residual as x and as y, out as y, beside each other in one buffer."""
    c = _case(dtype, "rms", "layer", 4, 0.9)
    y, x, gate, v = _inputs(21, width, c, True)
    (wr, tr), (wo, to) = block_norm64(y, x, gate, v, c)
    r, o, g = x.cuda(), y.cuda(), gate.cuda()
    _call(c, o, r, g, v, r, o)
    assert_within(r, wr, tr)
    assert_within(o, wo, to)
    r, o = y.cuda(), torch.empty_like(y, device="cuda")
    _call(c, r, x.cuda(), g, v, r, o)
    assert_within(r, wr, tr)
    assert_within(o, wo, to)
    wide = torch.full((21, 4 * width + 24), 7.0, dtype=y.dtype, device="cuda")
    parts = [wide[:, i * (width + 3):i * (width + 3) + width] for i in range(4)]
    parts[0].copy_(y)
    parts[1].copy_(x)
    s = wide.stride(0)
    _call(c, parts[0], parts[1], g, v, parts[2], parts[3], y_stride=s, x_stride=s, residual_stride=s, out_stride=s)
    assert_within(parts[2], wr, tr)
    assert_within(parts[3], wo, to)
    assert (wide[:, width:width + 3] == 7).all() and (wide[:, 4 * (width + 3):] == 7).all()
