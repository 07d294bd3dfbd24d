"""GPU: block_norm_forward of rows whose squares leave fp32's range, next to ordinary ones."""
import pytest
import torch

from attention_reference import TYPES, assert_within
from decoder_reference import block_norm64

pytestmark = pytest.mark.gpu


def _call(y, x, v, c):
    import convolution_conv2d_forward_amd as m
    d = m.block_norm_desc_create(m.make_block_norm_params(
        y.shape[1], post_norm=c["post"], pre_norm=c["pre"], has_post_beta=v[1] is not None, has_pre_beta=v[3] is not None,
        residual_scale=c["residual_scale"], block_scale=c["block_scale"], eps=c["eps"], dtype=c["dtype"]))
    r, o = torch.empty_like(y, device="cuda"), torch.empty_like(y, device="cuda")
    m.block_norm_forward(d, y.cuda(), x.cuda(), None, *(None if t is None else t.cuda() for t in v), r,
                         o if c["pre"] != "none" else None)
    return r, o


def _check(width, dtype, kind, scales, eps, where):
    """Row i is scaled by scales[i]; `where`: the norm that meets it."""
    g = torch.Generator().manual_seed(width)
    t, rows = TYPES[dtype], len(scales)
    base = torch.randn(rows, width, generator=g, dtype=torch.float64) + (0.5 if kind == "layer" else 0)
    far = (base * torch.tensor(scales, dtype=torch.float64)[:, None]).clamp(-3e38, 3e38).to(t)
    gamma, beta = 1 + 0.2 * torch.randn(width, generator=g), torch.randn(width, generator=g) if kind == "layer" else None
    c = dict(dtype=dtype, gate_rows=None, residual_scale=1.0, block_scale=1.0, eps=eps, post="none", pre="none")
    c[where] = kind
    v = [gamma, beta, None, None] if where == "post" else [None, None, gamma, beta]
    y, x = (far, torch.randn(rows, width, generator=g).to(t)) if where == "post" else (torch.zeros_like(far), far)
    got_r, got_o = _call(y, x, v, c)
    (r, tr), rest = block_norm64(y, x, None, v, c)
    assert_within(got_r, r, tr, "residual")
    if rest:
        assert_within(got_o, *rest, "out")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [64, 65, 1000, 4096, 8192, 8193, 16384, 20001, 32768])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("where", ["post", "pre"])
def test_large_rows(where, kind, width, dtype):
    """Squares beyond 3.4e38, sums of elements beyond it, elements at the border, ordinary rows between."""
    _check(width, dtype, kind, [1.0, 1e19, 1e20, 1.0, 1e30, 1e34, 1e37, 1e-3], 1e-6, where)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [64, 65, 4096, 9001, 32768])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("eps", [0.0, 1e-36])
def test_small_rows_without_an_eps(eps, kind, width, dtype):
    """Squares below 1.2e-38 where no eps outweighs them."""
    _check(width, dtype, kind, [1.0, 1e-18, 1e-20, 1e-25, 1.0, 1e-30, 1e3], eps, "post")


@pytest.mark.parametrize("width", [64, 65, 4096, 9001])
def test_bad_numbers_in_large_rows(width):
    """A row with an infinity or NaN stays one; its neighbours are as without it."""
    x = torch.full((3, width), 1e25)
    x[:, ::2] = -1e25
    x[1, 3] = float("inf")
    c = dict(dtype="f32", gate_rows=None, residual_scale=1.0, block_scale=1.0, eps=1e-6, post="none", pre="rms")
    _, o = _call(torch.zeros_like(x), x, [None, None, torch.ones(width), None], c)
    want = torch.where(torch.arange(width) % 2 == 0, -1.0, 1.0)
    assert torch.isnan(o[1, 3]) and ((o.cpu()[[0, 2]] - want).abs() <= (width + 8) * 2.0 ** -24).all()


@pytest.mark.parametrize("width", [3, 64, 999, 4096, 9001])
def test_elements_at_the_border_of_the_range(width):
    """Elements that are fp32's largest either way: an element less the mean, the mean's sum and the squares are beyond it."""
    big = torch.finfo(torch.float32).max
    x = torch.full((3, width), -big)
    x[0, 0] = big
    x[1] = big
    x[2, ::2] = big
    c = dict(dtype="f32", gate_rows=None, residual_scale=1.0, block_scale=1.0, eps=1e-6, post="none", pre="layer")
    _, o = _call(torch.zeros_like(x), x, [None, None, torch.ones(width), torch.zeros(width)], c)
    want = torch.where(x == big, 1.0, -1.0).double()
    want = want - want.mean(1, keepdim=True)
    spread = want.square().mean(1, keepdim=True).sqrt()
    off = (o.cpu().double()[[0, 2]] - (want / spread)[[0, 2]]).abs()
    assert (off <= 4 * (width + 8) * 2.0 ** -24 * (1 + (want / spread)[[0, 2]].abs()) / spread[[0, 2]]).all()
    assert torch.isfinite(o).all()   # a row without spread is rounding alone
