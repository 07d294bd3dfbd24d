"""GPU: linear_forward's activations at infinities and far into their tails."""
import math

import pytest
import torch

from attention_reference import FN, ROUND, TYPES, U32

pytestmark = pytest.mark.gpu


def cc():
    import convolution_conv2d_forward_amd as m
    return m


def _apply(values, act, dtype, m, n=24, k=64, **kw):
    """act of each value: x has the value in its row's first place and zeros
    after it, w is all ones.  values fill m rows in turn; [m, n] on the CPU."""
    x = torch.zeros(m, k, dtype=TYPES[dtype])
    x[:, 0] = torch.tensor([values[i % len(values)] for i in range(m)]).to(TYPES[dtype])
    d = cc().linear_desc_create(cc().make_linear_params(k, n, act=act, dtype=dtype, **kw))
    y = torch.empty(m, n, dtype=TYPES[dtype], device="cuda")
    cc().linear_forward(d, x.cuda(), torch.ones(n, k, dtype=TYPES[dtype], device="cuda"), None, None, y)
    y = y.cpu()
    assert torch.equal(torch.nan_to_num(y, 7.0), torch.nan_to_num(y[:, :1].expand(m, n), 7.0)), "columns differ"
    return x[:, 0].double(), y[:, 0].double()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [1, 40, 300])
@pytest.mark.parametrize("act,want", [("none", math.inf), ("relu", math.inf), ("leaky_relu", math.inf), ("clip", 0.75),
                                      ("silu", math.inf), ("gelu", math.inf), ("gelu_tanh", math.inf)])
def test_plus_infinity(act, want, m, dtype):
    _, y = _apply([math.inf], act, dtype, m, **({"clip": (-0.5, 0.75)} if act == "clip" else {}))
    assert (y == want).all()


TAIL = [-0.01 * 1.09 ** i for i in range(77)] + [0.02 * 1.1 ** i for i in range(70)]   # to -7 and 14


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [9, 147, 300])
def test_gelu_tanh_keeps_its_relative_accuracy(m, dtype):
    """v / (1 + exp(-2 u)), u = sqrt(2/pi) (v + 0.044715 v^3).  u is off by
    4 roundings, which the exponential multiplies by 2 |u|; itself it is off by
    2^-21 and, as a power of two, by the rounding of an argument 2 |u| log2 e."""
    v, y = _apply(TAIL, "gelu_tanh", dtype, m)
    u = math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
    want = v / (1 + torch.exp(-2 * u))
    rel = 2 * u.abs() * 8 * U32 + FN + 8 * U32 + ROUND[dtype]
    over = (y - want).abs() / want.abs() / rel
    assert (over <= 1).all(), (float(v[over.argmax()]), float(over.max()))


@pytest.mark.parametrize("m", [9, 147, 300])
def test_silu_keeps_its_relative_accuracy(m):
    """fp32: v / (1 + exp(-v)), the exponential and the quotient off by 2^-21
    together, down to -85, where it is 1e-35."""
    v, y = _apply([-0.01 * 1.064 ** i for i in range(147)], "silu", "f32", m)
    want = v / (1 + torch.exp(-v))
    over = (y - want).abs() / want.abs() / (FN + 4 * U32)
    assert (over <= 1).all(), (float(v[over.argmax()]), float(over.max()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [9, 147, 300])
def test_gelu_keeps_its_relative_accuracy(m, dtype):
    """v erfc(-v / sqrt 2) / 2: the argument z is off by 2 roundings, which
    erfc multiplies by up to 2 z^2 + 1; the function by 2^-21."""
    v, y = _apply(TAIL, "gelu", dtype, m)
    want = 0.5 * v * torch.special.erfc(-v / math.sqrt(2))
    rel = (v * v + 1) * 2 * U32 + FN + 8 * U32 + ROUND[dtype]
    over = (y - want).abs() / want.abs() / rel
    assert (over <= 1).all(), (float(v[over.argmax()]), float(over.max()))
