"""GPU: linear_forward against the 64-bit definition, at sizes around the
kernels' tiles, odd sizes, strides, activations, in-place residuals."""
import pytest
import torch

from attention_reference import TYPES, assert_within, linear64

pytestmark = pytest.mark.gpu


def cc():
    import convolution_conv2d_forward_amd as m
    return m


def _inputs(m, k, n, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g).to(TYPES[dtype])
    w = (torch.randn(n, k, generator=g) * k ** -0.5).to(TYPES[dtype])
    return x, w, torch.randn(n, generator=g), torch.randn(m, n, generator=g).to(TYPES[dtype])


def _run(m, k, n, dtype, act="none", bias=True, residual=True, seed=0, **kw):
    x, w, b, r = _inputs(m, k, n, dtype, seed)
    d = cc().linear_desc_create(cc().make_linear_params(k, n, has_bias=bias, has_residual=residual, act=act,
                                                        dtype=dtype, **kw))
    y = torch.full((m, n), float("nan"), dtype=TYPES[dtype], device="cuda")
    cc().linear_forward(d, x.cuda(), w.cuda(), b.cuda() if bias else None, r.cuda() if residual else None, y)
    want, tol = linear64(x, w, b if bias else None, r if residual else None, dtype, act, kw.get("alpha") or 0.01,
                         kw.get("clip") or (-float("inf"), float("inf")))
    assert_within(y, want, tol, f"{m}x{k}x{n} {dtype} {act} [{cc().linear_desc_kernel_name(d, m)}]")


SIZES = [(1, 1, 1), (1, 8, 4), (2, 64, 16), (3, 7, 5), (1, 1024, 1536), (1, 1000, 777), (4, 4096, 64), (8, 96, 100),
         (15, 640, 48), (16, 512, 512), (17, 130, 33), (24, 2048, 1000), (31, 72, 200), (33, 4096, 64), (48, 264, 96),
         (64, 64, 64), (65, 192, 130), (100, 8192, 40), (127, 128, 129), (130, 96, 258), (256, 256, 256),
         (300, 520, 264), (257, 1024, 513), (515, 200, 768), (1024, 512, 1024), (1571, 770, 300)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,k,n", SIZES)
def test_sizes(m, k, n, dtype):
    _run(m, k, n, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,k,n", [(2, 96, 72), (40, 130, 70), (200, 256, 320)])
@pytest.mark.parametrize("act", ["none", "relu", "leaky_relu", "clip", "silu", "gelu", "gelu_tanh"])
def test_activations(act, m, k, n, dtype):
    kw = {"alpha": 0.2} if act == "leaky_relu" else {"clip": (-0.5, 0.75)} if act == "clip" else {}
    _run(m, k, n, dtype, act, **kw)


@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("m", [1, 20, 300])
def test_without_bias_or_residual(m, bias, residual):
    _run(m, 256, 136, "bf16", "gelu", bias, residual)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [1, 9, 140])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_strided_rows_inside_wider_buffers(m, shift, dtype):
    """x, the residual and y are column slices; the columns next to y keep
    their values, and an in-place residual is the same call with y = residual."""
    k, n, t = 200, 152, TYPES[dtype]
    x, w, b, r = _inputs(m, k, n, dtype, 5)
    wide_x = torch.full((m, k + 24), float("nan"), dtype=t, device="cuda")
    wide_y = torch.full((m, n + 40), 7.0, dtype=t, device="cuda")
    xv, yv = wide_x[:, shift:shift + k], wide_y[:, shift:shift + n]
    xv.copy_(x)
    yv.copy_(r)
    d = cc().linear_desc_create(cc().make_linear_params(k, n, has_bias=True, has_residual=True, act="silu",
                                                        x_stride=k + 24, y_stride=n + 40, residual_stride=n + 40,
                                                        dtype=dtype))
    cc().linear_forward(d, xv, w.cuda(), b.cuda(), yv, yv)
    want, tol = linear64(x, w, b, r, dtype, "silu")
    assert_within(yv, want, tol)
    assert (wide_y[:, :shift] == 7).all() and (wide_y[:, shift + n:] == 7).all()


def test_rows_beyond_32_bit_offsets():
    m, k, n, stride = 5, 64, 32, (1 << 30) + 8
    buf = torch.empty((m - 1) * stride + k, dtype=torch.bfloat16, device="cuda")
    x, w, b, r = _inputs(m, k, n, "bf16", 3)
    xv = buf.as_strided((m, k), (stride, 1))
    xv.copy_(x)
    d = cc().linear_desc_create(cc().make_linear_params(k, n, x_stride=stride, dtype="bf16"))
    y = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    cc().linear_forward(d, xv, w.cuda(), None, None, y)
    want, tol = linear64(x, w, None, None, "bf16")
    assert_within(y, want, tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [2, 200])
def test_infinities_and_nan_stay_in_their_rows(m, dtype):
    k, n = 128, 96
    x, w, _, _ = _inputs(m, k, n, dtype, 9)
    x[1, 5] = float("inf")
    w[3, 7] = float("nan")
    d = cc().linear_desc_create(cc().make_linear_params(k, n, dtype=dtype))
    y = torch.empty((m, n), dtype=TYPES[dtype], device="cuda")
    cc().linear_forward(d, x.cuda(), w.cuda(), None, None, y)
    got = y.cpu().double()
    want = x.double() @ w.double().T
    assert torch.isnan(got[:, 3]).all()
    assert torch.isinf(got[1, [c for c in range(n) if c != 3]]).all()
    fine = torch.isfinite(want)
    assert torch.isfinite(got[fine]).all()


def test_no_rows_launches_nothing_and_same_results_twice():
    d = cc().linear_desc_create(cc().make_linear_params(64, 64, dtype="bf16"))
    w = torch.randn(64, 64, device="cuda").bfloat16()
    cc().linear_forward(d, torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), w, None, None,
                        torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    for m in (1, 30, 700):
        x = torch.randn(m, 64, device="cuda").bfloat16()
        ys = [torch.empty((m, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        for y in ys:
            cc().linear_forward(d, x, w, None, None, y)
        assert torch.equal(*ys)
