"""Host-only tests of include/attention.h: exports, struct layouts, defaults,
refusals before any launch, and the 64-bit reference's masks by hand."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

from attention_reference import seen

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "attention.h")


def cc():
    import convolution_conv2d_forward_amd as m
    return m


def att():
    from convolution_conv2d_forward_amd import attention as m
    return m


def test_header_symbols_exported():
    syms = sorted(set(re.findall(r"CONV2D_API\s+[\w\s\*]+?\b(\w+)\s*\(", open(HEADER).read())))
    assert sorted(att().EXPORTED) == syms
    lib = ctypes.CDLL(cc().LIB_PATH)
    for s in syms:
        assert hasattr(lib, s), s


@pytest.mark.parametrize("name", ["linear_params_t", "qk_rope_params_t", "attention_params_t"])
def test_params_layout_matches_header(tmp_path, name):
    P = getattr(cc(), name)
    names = [f[0] for f in P._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "%s"\nint main(void) {\n'
                   '  printf("%%zu\\n", sizeof(%s));\n%s  return 0;\n}\n'
                   % (HEADER, name, "".join('  printf("%%zu\\n", offsetof(%s, %s));\n' % (name, n) for n in names)))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", str(src), "-o", str(exe)], check=True)
    out = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert out[0] == ctypes.sizeof(P)
    assert out[1:] == [getattr(P, n).offset for n in names]


def _status(create, make, *a, **kw):
    with pytest.raises(cc().ConvError) as e:
        create(make(*a, **kw))
    assert cc().conv2d_last_error()
    return e.value.status


def test_linear_desc_refusals():
    m = cc()
    bad = lambda *a, **kw: _status(m.linear_desc_create, m.make_linear_params, *a, **kw)  # noqa: E731
    inv, shapes, uns = m.CONV_ERR_INVALID_ARG, m.CONV_ERR_INCOMPATIBLE_SHAPES, m.CONV_ERR_UNSUPPORTED
    assert bad(0, 4) == inv and bad(4, 0) == inv and bad(-1, 4) == inv and bad((1 << 24) + 1, 4) == inv
    assert bad(8, 8, dtype="i8") == uns and bad(8, 8, dtype=9) == inv
    assert bad(8, 8, act=m.ACT_PRELU) == uns and bad(8, 8, act=99) == inv
    assert bad(8, 8, act="clip", clip=(1.0, 0.0)) == inv and bad(8, 8, act="leaky_relu", alpha=math.inf) == inv
    assert bad(8, 8, x_stride=7) == shapes and bad(8, 8, y_stride=-8) == inv and bad(8, 8, residual_stride=3) == shapes
    assert m._lib.linear_desc_create(None, None) == inv


def test_linear_call_refusals():
    m = cc()
    d = m.linear_desc_create(m.make_linear_params(16, 8, has_bias=True, has_residual=True, x_stride=32, y_stride=32,
                                                  residual_stride=32))
    f = lambda *a: m._lib.linear_forward(d.handle, *a, None)  # noqa: E731
    x, w, b, r, y = (4096 * i for i in (100, 200, 300, 400, 500))
    inv, alias = m.CONV_ERR_INVALID_ARG, m.CONV_ERR_ALIAS
    assert f(-1, x, w, b, r, y) == inv and f(1 << 31, x, w, b, r, y) == inv
    assert f(4, None, w, b, r, y) == inv and f(4, x, None, b, r, y) == inv and f(4, x, w, None, r, y) == inv
    assert f(4, x, w, b, None, y) == inv and f(4, x, w, b, r, None) == inv
    assert f(4, x + 2, w, b, r, y) == inv and f(4, x, w, b + 1, r, y) == inv
    assert f(4, x, w, b, r, x + 60) == alias          # rows 0..15 of x against 8 columns from 15 on
    assert f(4, x, w, b, r, w + 128) == alias and f(4, x, w, b, r, b + 4) == alias
    assert f(4, x, w, b, r, r + 4) == alias           # shifted against the residual
    assert f(0, None, None, None, None, None) == m.CONV_OK
    assert m._lib.linear_forward(None, 1, x, w, b, r, y, None) == inv
    assert m.linear_desc_kernel_name(d, 5) and m._lib.linear_desc_kernel_name(None, 5) == b""


def test_qk_rope_refusals():
    m = cc()
    bad = lambda *a, **kw: _status(m.qk_rope_desc_create, m.make_qk_rope_params, *a, **kw)  # noqa: E731
    inv, shapes, uns = m.CONV_ERR_INVALID_ARG, m.CONV_ERR_INCOMPATIBLE_SHAPES, m.CONV_ERR_UNSUPPORTED
    assert bad(0, 1, 64) == inv and bad(1, 0, 64) == inv and bad(1, 1, 0) == inv and bad(1, 1, 258) == uns
    assert bad(1, 1, 7) == inv and bad(1, 1, 8, rotary_dim=3) == inv and bad(1, 1, 8, rotary_dim=10) == shapes
    assert bad(1, 1, 8, layout=2) == inv and bad(1, 1, 8, scaling=3) == inv and bad(1, 1, 8, eps=-1.0) == inv
    assert bad(1, 1, 8, theta=1.0) == inv and bad(1, 1, 8, factor=0.5) == inv and bad(1, 1, 8, theta=math.nan) == inv
    assert bad(1, 1, 8, scaling="yarn", factor=2.0) == inv and bad(1, 1, 8, attn_factor=-1.0) == inv
    assert bad(1, 1, 8, scaling="yarn", factor=2.0, original_len=64, beta_fast=0.0) == inv
    assert bad(1, 1, 8, qkv_stride=23) == shapes and bad(2, 1, 8, q_stride=8) == shapes and bad(1, 1, 8, dtype="i8") == uns
    d = m.qk_rope_desc_create(m.make_qk_rope_params(2, 1, 8, has_norm=True))
    f = lambda *a: m._lib.qk_rope_forward(d.handle, *a, None)  # noqa: E731
    qkv, gq, gk, pos, sl, q, k, v = (4096 * i for i in range(100, 900, 100))
    alias = m.CONV_ERR_ALIAS
    assert f(-1, qkv, gq, gk, pos, sl, 9, q, k, v) == inv and f(4, qkv, gq, gk, pos, sl, -1, q, k, v) == inv
    assert f(4, None, gq, gk, pos, sl, 9, q, k, v) == inv and f(4, qkv, None, gk, pos, sl, 9, q, k, v) == inv
    assert f(4, qkv, gq, gk, None, sl, 9, q, k, v) == inv and f(4, qkv, gq, gk, pos, sl, 9, q, None, v) == inv
    assert f(4, qkv, gq, gk, pos, None, 3, q, k, v) == shapes
    assert f(4, qkv + 2, gq, gk, pos, sl, 9, q, k, v) == inv and f(4, qkv, gq, gk, pos + 1, sl, 9, q, k, v) == inv
    assert f(4, qkv, gq, gk, pos, sl, 9, qkv + 4, k, v) == alias and f(4, qkv, gq, gk, pos, sl, 9, qkv, k, v) == alias
    assert f(4, qkv, gq, gk, pos, sl, 9, q, qkv, v) == alias and f(4, qkv, gq, gk, pos, sl, 9, q, k, k + 32) == alias
    assert f(4, qkv, gq, gk, pos, sl, 9, q, q + 32, v) == alias and f(4, qkv, gq, gk, pos, sl, 9, pos, k, v) == alias
    assert f(0, None, None, None, None, None, 0, None, None, None) == m.CONV_OK


def _strides(d=64, h=4, **kw):
    s = {n: (h * d * 100, h * d, d) for n in ("q_strides", "k_strides", "v_strides", "out_strides")}
    s.update(kw)
    return s


def test_attention_refusals():
    m = cc()
    bad = lambda *a, **kw: _status(m.attention_desc_create, m.make_attention_params, *a, **{**_strides(), **kw})  # noqa: E731
    inv, shapes, uns = m.CONV_ERR_INVALID_ARG, m.CONV_ERR_INCOMPATIBLE_SHAPES, m.CONV_ERR_UNSUPPORTED
    assert bad(0, 1, 64) == inv and bad(4, 3, 64) == shapes and bad(4, 2, 0) == inv
    assert bad(4, 2, 264) == uns and bad(4, 2, 62) == uns and bad(4, 2, 60, dtype="bf16") == uns
    assert bad(4, 2, 64, dtype="i8") == uns and bad(4, 2, 64, window=-1) == inv
    assert bad(4, 2, 64, softcap=-1.0) == inv and bad(4, 2, 64, softcap=math.nan) == inv and bad(4, 2, 64, scale=math.inf) == inv
    assert bad(4, 2, 64, k_strides=(-64, 64, 64)) == inv and bad(4, 2, 64, q_strides=(0, 66, 64)) == uns
    assert bad(4, 2, 64, out_strides=(6400, 64, 0)) == shapes
    d = m.attention_desc_create(m.make_attention_params(4, 2, 64, has_slopes=True, **_strides()))
    g = lambda *a: m._lib.attention_forward(d.handle, *a, None)  # noqa: E731
    P = 1 << 24
    q, k, v, o, ws, s = (P * i for i in range(1, 7))
    big = 1 << 20
    assert g(-1, 1, 9, q, k, v, None, None, None, None, 0, s, o, ws, big) == inv
    assert g(1, 1, (1 << 30) + 1, q, k, v, None, None, None, None, 0, s, o, ws, big) == inv
    assert g(1, 1, 9, None, k, v, None, None, None, None, 0, s, o, ws, big) == inv
    assert g(1, 1, 9, q, None, v, None, None, None, None, 0, s, o, ws, big) == inv
    assert g(1, 1, 9, q + 8, k, v, None, None, None, None, 0, s, o, ws, big) == inv
    assert g(1, 1, 9, q, k, v, q + 2, None, None, None, 0, s, o, ws, big) == inv
    assert g(1, 1, 9, q, k, v, None, None, None, None, 0, None, o, ws, big) == inv
    assert g(1, 1, 9, q, k, v, None, None, None, s + 64, 0, s, o, ws, big) == inv
    assert g(1, 1, 9, q, k, v, None, None, None, None, 0, s, q, ws, big) == m.CONV_ERR_ALIAS
    need = m.attention_workspace_bytes(d, 1, 1, 5000)
    assert need > 0
    assert g(1, 1, 5000, q, k, v, None, None, None, None, 0, s, o, ws, need - 1) == inv
    assert g(1, 1, 5000, q, k, v, None, None, None, None, 0, s, o, None, need) == inv
    assert g(1, 1, 5000, q, k, v, None, None, None, None, 0, s, o, o, need) == m.CONV_ERR_ALIAS
    assert g(1, 1, 5000, q, k, v, None, None, None, None, 0, s, o, k, need) == m.CONV_ERR_ALIAS
    assert g(0, 1, 9, None, None, None, None, None, None, None, 0, None, None, None, 0) == m.CONV_OK
    assert m.attention_workspace_bytes(d, 0, 1, 5000) == 0
    with pytest.raises(m.ConvError):
        m.attention_workspace_bytes(d, 1, -1, 5)
    far = m.attention_desc_create(m.make_attention_params(4, 2, 64, **_strides(k_strides=(1 << 40, 1 << 40, 64))))
    assert m._lib.attention_forward(far.handle, 64, 1, 64, q, k, v, None, None, None, None, 0, None, o, ws, big,
                                    None) == uns


def test_binding_refusals():
    """The binding names a wrong tensor before the library is called."""
    m = cc()
    d = m.linear_desc_create(m.make_linear_params(8, 8))
    x = torch.zeros(2, 8)
    with pytest.raises(TypeError):
        m.linear_forward(d, x, x, None, None, x)


def test_reference_masks_by_hand():
    s = lambda *a, **kw: seen(*a, **{"causal": False, "window": 0, "prefix": None, "docs": None, **kw}).int().tolist()  # noqa: E731
    assert s(2, 3, 2, 3, causal=True) == [[1, 1, 0], [1, 1, 1]]
    assert s(3, 2, 3, 2, causal=True) == [[0, 0], [1, 0], [1, 1]]
    assert s(2, 4, 2, 4, causal=True, prefix=4) == [[1, 1, 1, 1]] * 2
    assert s(1, 4, 1, 3, window=2) == [[0, 1, 1, 0]]
    assert s(3, 3, 3, 3, docs=[0, 1, 3]) == [[1, 0, 0], [0, 1, 1], [0, 1, 1]]
    assert s(3, 3, 2, 2, causal=True) == [[1, 0, 0], [1, 1, 0], [0, 0, 0]]


def test_attention_grids_beyond_a_launch():
    """A launch holds 2^24 - 1 workgroups of 256 threads: many sequences may take
    several, one sequence has to fit."""
    m = cc()
    s = (1 << 20, 1 << 10, 8)
    d = m.attention_desc_create(m.make_attention_params(128, 128, 8, dtype="bf16", q_strides=s, k_strides=s, v_strides=s,
                                                        out_strides=s))
    assert m.attention_workspace_bytes(d, 1 << 20, 1, 1) == 0        # 2^27 workgroups
    assert m.attention_workspace_bytes(d, 1, (1 << 24) - 128, 1) == 0   # 2^24 - 128 tiles of 128 rows
    with pytest.raises(m.ConvError) as e:
        m.attention_workspace_bytes(d, 1, 1 << 24, 1)
    assert e.value.status == m.CONV_ERR_UNSUPPORTED
    P = 1 << 40
    assert m._lib.attention_forward(d.handle, 1, 1 << 24, 1, P, 2 * P, 3 * P, None, None, None, None, 0, None, 4 * P, None, 0,
                                    None) == m.CONV_ERR_UNSUPPORTED


@pytest.mark.parametrize("rows", [(1 << 31) - 1, (1 << 31) - 15, (1 << 31) - 64])
@pytest.mark.parametrize("k,n,dtype", [(1, 1, "bf16"), (8, 8, "bf16"), (4096, 16, "f32"), (8, 1 << 24, "f32")])
def test_linear_rule_at_the_most_rows(k, n, dtype, rows):
    """Roundings of the row count stay within their type: so many rows go to
    tiles, or, where k is long, to workgroups of 64 rows."""
    m = cc()
    d = m.linear_desc_create(m.make_linear_params(k, n, dtype=dtype))
    assert m.linear_desc_kernel_name(d, rows) == m.linear_desc_kernel_name(d, 1 << 28)


@pytest.mark.parametrize("strides,status", [
    ((6400, 64, 64), "ALIAS"), ((64, 256, 64), "ALIAS"), ((640, 256, 64), "ALIAS"), ((6400, 128, 64), "ALIAS"),
    ((6400, 64, 128), "ALIAS"),                                   # a token's heads 0 and 1 are 2 tokens apart
    ((1280, 256, 64), "OK"), ((256, 512, 64), "OK"), ((1280, 64, 320), "OK"), ((1600, 320, 80), "OK"),
], ids=str)
def test_attention_rows_of_out_share_no_memory(strides, status):
    """2 sequences, 5 tokens, 4 heads of 64.  Accepted ones go on to the check of
    the workspace, which follows."""
    m = cc()
    d = m.attention_desc_create(m.make_attention_params(4, 4, 64, **_strides(out_strides=strides)))
    P = 1 << 30
    status_of = lambda ws: m._lib.attention_forward(  # noqa: E731
        d.handle, 2, 5, 5000, P, 2 * P, 3 * P, None, None, None, None, 0, None, 4 * P, ws, 1 << 30, None)
    need = m.attention_workspace_bytes(d, 2, 5, 5000)
    assert need > 0
    assert status_of(4 * P) == m.CONV_ERR_ALIAS
    assert ("share" in m.conv2d_last_error()) == (status == "ALIAS"), m.conv2d_last_error()
