"""Host-only tests of include/decoder.h: exports, struct layouts, refusals before any launch, and the 64-bit
reference by hand."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

from decoder_reference import E4M3, quantise64, seen64

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "decoder.h")


def cc():
    import convolution_conv2d_forward_amd as m
    return m


def test_header_symbols_exported():
    from convolution_conv2d_forward_amd import decoder
    syms = sorted(set(re.findall(r"CONV2D_API\s+[\w\s\*]+?\b(\w+)\s*\(", open(HEADER).read())))
    assert sorted(decoder.EXPORTED) == syms
    lib = ctypes.CDLL(cc().LIB_PATH)
    for s in syms:
        assert hasattr(lib, s), s


@pytest.mark.parametrize("name", ["kv_cache_params_t", "paged_attention_params_t", "block_norm_params_t"])
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


P = 1 << 30   # far from each other, 16-byte aligned


def test_kv_cache_refusals():
    m = cc()
    bad = lambda *a, **kw: _status(m.kv_cache_desc_create, m.make_kv_cache_params, *a, **kw)  # noqa: E731
    inv, shapes, uns, alias = m.CONV_ERR_INVALID_ARG, m.CONV_ERR_INCOMPATIBLE_SHAPES, m.CONV_ERR_UNSUPPORTED, m.CONV_ERR_ALIAS
    assert bad(0, 64, 16) == inv and bad(1, 0, 16) == inv and bad(1, 257, 16) == uns and bad((1 << 16) + 1, 8, 1) == inv
    assert bad(1, 64, 0) == inv and bad(1, 64, (1 << 16) + 1) == inv
    assert bad(1, 64, 16, dtype="i8") == uns and bad(1, 64, 16, dtype="f32", cache_dtype="bf16") == uns
    assert bad(1, 64, 16, cache_dtype="i8") == uns and bad(1, 64, 16, cache_dtype=17) == inv and bad(1, 64, 16, dtype=16) == inv
    assert bad(2, 64, 16, k_stride=127) == shapes and bad(2, 64, 16, v_stride=-128) == inv and bad(2, 64, 16, k_batch_stride=-1) == inv
    assert bad(2, 64, 16, k_page_strides=(2048, 64, 63)) == shapes and bad(2, 64, 16, scale_strides=(16, 0, 1)) == shapes
    assert bad(2, 64, 16, v_page_strides=(-1, 64, 64)) == inv and m._lib.kv_cache_desc_create(None, None) == inv
    d = m.kv_cache_desc_create(m.make_kv_cache_params(2, 64, 16, dtype="bf16", cache_dtype="e4m3"))
    f = lambda *a: m._lib.kv_cache_store(d.handle, *a, None)  # noqa: E731
    k, v, sl, kp, vp, ks, vs = (P * i for i in range(1, 8))
    assert f(-1, k, v, sl, 9, kp, vp, ks, vs) == inv and f(4, k, v, sl, -1, kp, vp, ks, vs) == inv
    assert f(4, k, v, sl, 1 << 27, kp, vp, ks, vs) == inv and f(1 << 31, k, v, sl, 9, kp, vp, ks, vs) == inv
    for i in (0, 1, 2, 4, 5, 6, 7):
        args = [k, v, sl, 9, kp, vp, ks, vs]
        args[i] = None
        assert f(4, *args) == inv, i
    assert f(4, k + 1, v, sl, 9, kp, vp, ks, vs) == inv and f(4, k, v, sl + 2, 9, kp, vp, ks, vs) == inv
    assert f(4, k, v, sl, 9, k + 100, vp, ks, vs) == alias and f(4, k, v, sl, 9, kp, kp + 64, ks, vs) == alias
    assert f(4, k, v, sl, 9, kp, vp, ks, ks + 1) == alias and f(4, k, v, sl, 9, kp, vp, ks, sl) == alias
    assert f(4, k, v, sl, 9, kp, vp, kp + 5, vs) == alias
    assert f(0, None, None, None, 9, None, None, None, None) == m.CONV_OK
    assert m._lib.kv_cache_store(None, 4, k, v, sl, 9, kp, vp, ks, vs, None) == inv
    shared = m.kv_cache_desc_create(m.make_kv_cache_params(2, 64, 16, dtype="bf16", k_page_strides=(64, 64, 64)))
    assert m._lib.kv_cache_store(shared.handle, 4, k, v, sl, 9, kp, vp, None, None, None) == alias
    far = m.kv_cache_desc_create(m.make_kv_cache_params(2, 64, 16, k_page_strides=(1 << 40, 128, 64)))
    assert m._lib.kv_cache_store(far.handle, 4, k, v, sl, 99, kp, vp, None, None, None) == uns
    # Keys and values of a page beside each other in one buffer are no overlap.
    pair = m.kv_cache_desc_create(m.make_kv_cache_params(2, 64, 16, dtype="bf16", k_page_strides=(4096, 128, 64),
                                                         v_page_strides=(4096, 128, 64)))
    assert m._lib.kv_cache_store(pair.handle, 4, k, v, kp, 9, kp, kp + 2 * 2048, None, None, None) == alias
    assert "input" in m.conv2d_last_error()
    g = lambda *a: m._lib.kv_cache_load(d.handle, *a, None)  # noqa: E731
    t, n = P * 8, P * 9
    assert g(-1, 5, 5, t, n, 9, kp, vp, ks, vs, k, v) == inv and g(2, 5, 1 << 27, t, n, 9, kp, vp, ks, vs, k, v) == inv
    assert g(2, 5, 5, None, n, 9, kp, vp, ks, vs, k, v) == inv and g(2, 5, 5, t, n + 1, 9, kp, vp, ks, vs, k, v) == inv
    assert g(2, 5, 5, t, n, 9, kp, vp, None, vs, k, v) == inv and g(2, 5, 5, t, n, 9, kp, vp, ks, vs, None, v) == inv
    assert g(2, 5, 5, t, n, 9, kp, vp, ks, vs, k, k + 128) == alias and g(2, 5, 5, t, n, 9, kp, vp, ks, vs, kp, v) == alias
    assert g(2, 5, 5, t, n, 9, kp, vp, ks, vs, t, v) == alias and g(2, 5, 5, t, n, 9, kp, vp, ks, vs, ks, v) == alias
    assert g(0, 5, 5, None, None, 9, None, None, None, None, None, None) == m.CONV_OK
    both = m.kv_cache_desc_create(m.make_kv_cache_params(2, 64, 16, dtype="bf16", k_batch_stride=128))
    assert m._lib.kv_cache_load(both.handle, 2, 5, 5, t, n, 9, kp, vp, None, None, k, v, None) == alias


def test_paged_attention_refusals():
    m = cc()
    bad = lambda *a, **kw: _status(m.paged_attention_desc_create, m.make_paged_attention_params, *a, **kw)  # noqa: E731
    inv, shapes, uns, alias = m.CONV_ERR_INVALID_ARG, m.CONV_ERR_INCOMPATIBLE_SHAPES, m.CONV_ERR_UNSUPPORTED, m.CONV_ERR_ALIAS
    assert bad(0, 1, 64, 16) == inv and bad(4, 3, 64, 16) == shapes and bad(4, 2, 0, 16) == inv and bad(4, 2, 64, 0) == inv
    assert bad(4, 2, 264, 16) == uns and bad(4, 2, 62, 16) == uns and bad(4, 2, 60, 16, dtype="bf16") == uns
    assert bad(4, 2, 20, 16, cache_dtype="e4m3") == uns and bad(4, 2, 72, 16, dtype="bf16", cache_dtype="e4m3") == uns
    assert bad(4, 2, 64, 16, dtype="bf16", cache_dtype="e4m3", k_page_strides=(2056, 128, 64)) == uns
    assert bad(4, 2, 64, 16, dtype="bf16", cache_dtype="f32") == uns
    assert bad(4, 2, 64, 16, window=-1) == inv and bad(4, 2, 64, 16, sinks=-1) == inv and bad(4, 2, 64, 16, softcap=-1.0) == inv
    assert bad(4, 2, 64, 16, softcap=math.nan) == inv and bad(4, 2, 64, 16, scale=math.inf) == inv
    assert bad(4, 2, 64, 16, q_stride=255) == shapes and bad(4, 2, 64, 16, q_stride=258) == uns
    assert bad(4, 2, 64, 16, k_page_strides=(2050, 128, 64)) == uns and bad(4, 2, 64, 16, v_page_strides=(-2048, 128, 64)) == inv
    d = m.paged_attention_desc_create(m.make_paged_attention_params(4, 2, 64, 16, dtype="bf16", cache_dtype="e4m3"))
    need = m.paged_attention_workspace_bytes(d, 2, 2, 500)
    q, off, kv, tab, kp, vp, ks, vs, out, ws = (P * i for i in range(1, 11))
    big = max(need, 1 << 20)

    def f(tokens=2, batch=2, max_pages=500, q=q, off=off, kv=kv, tab=tab, n_pages=1000, kp=kp, vp=vp, ks=ks, vs=vs, out=out, ws=ws, n=big, d=d):
        return m._lib.paged_attention_forward(d.handle if d else None, tokens, batch, max_pages, q, off, kv, tab, n_pages,
                                              kp, vp, ks, vs, out, ws, n, None)
    assert f(tokens=-1) == inv and f(batch=-1) == inv and f(max_pages=-1) == inv and f(n_pages=-1) == inv and f(d=None) == inv
    assert f(max_pages=1 << 27) == inv and f(tokens=1 << 30) == uns and f(n_pages=1 << 27) == inv
    for name in ("q", "off", "kv", "tab", "kp", "vp", "ks", "vs", "out"):
        assert f(**{name: None}) == inv, name
    assert f(q=q + 8) == inv and f(kp=kp + 8) == inv and f(off=off + 2) == inv and f(ws=ws + 8) == inv
    assert f(out=q) == alias and f(out=off) == alias and f(out=ks) == alias and f(out=kp + 64) == alias
    assert f(tokens=0, q=None, out=None) == m.CONV_OK and f(batch=0, off=None) == m.CONV_OK
    if need:
        assert f(n=need - 1) == inv and f(ws=None) == inv and f(ws=out) == alias and f(ws=kv) == alias
    wide = m.paged_attention_desc_create(m.make_paged_attention_params(
        4, 2, 64, 16, dtype="bf16", cache_dtype="e4m3", k_page_strides=(1 << 36, 128, 64)))
    assert f(d=wide) == uns
    with pytest.raises(m.ConvError):
        m.paged_attention_workspace_bytes(d, 1, -1, 5)
    assert m.paged_attention_workspace_bytes(d, 0, 3, 5) == 0


def test_block_norm_refusals():
    m = cc()
    bad = lambda *a, **kw: _status(m.block_norm_desc_create, m.make_block_norm_params, *a, **kw)  # noqa: E731
    inv, shapes, uns, alias = m.CONV_ERR_INVALID_ARG, m.CONV_ERR_INCOMPATIBLE_SHAPES, m.CONV_ERR_UNSUPPORTED, m.CONV_ERR_ALIAS
    assert bad(0) == inv and bad(32769) == uns and bad(8, dtype="i8") == uns and bad(8, post_norm=3) == inv
    assert bad(8, pre_norm=-1) == inv and bad(8, has_post_beta=True) == inv and bad(8, gate_rows=-1) == inv
    assert bad(8, residual_scale=math.nan) == inv and bad(8, block_scale=math.inf) == inv and bad(8, eps=-1.0) == inv
    assert bad(8, y_stride=7) == shapes and bad(8, gate_stride=-8) == inv
    d = m.block_norm_desc_create(m.make_block_norm_params(16, post_norm="rms", pre_norm="layer", has_pre_beta=True,
                                                          has_gate=True, gate_rows=3))
    y, x, g, pg, pb, qg, qb, r, o = (P * i for i in range(1, 10))

    def f(rows=7, y=y, x=x, g=g, pg=pg, pb=None, qg=qg, qb=qb, r=r, o=o):
        return m._lib.block_norm_forward(d.handle, rows, y, x, g, pg, pb, qg, qb, r, o, None)
    assert f(rows=-1) == inv and f(rows=1 << 31) == inv
    for name in ("y", "x", "g", "pg", "qg", "qb", "r", "o"):
        assert f(**{name: None}) == inv, name
    assert f(y=y + 2) == inv and f(pg=pg + 1) == inv
    assert f(r=x + 64) == alias and f(r=y + 64) == alias and f(o=x) == alias and f(o=y + 4) == alias and f(o=r) == alias
    assert f(r=g + 2 * 64) == alias and f(o=qg) == alias and f(r=y, o=y) == alias
    assert f(rows=0, y=None) == m.CONV_OK


def test_tensors_of_no_gpu_are_refused():
    """The binding's check of a call's tensors: none of them may lie elsewhere than on the call's device."""
    cc()
    from convolution_conv2d_forward_amd._marshal import on_device
    x = torch.zeros(2, 8)
    with pytest.raises((ValueError, TypeError), match="x"):
        on_device(0, x, "x", torch.float32, (2, 8), None)
    for args in ((x, "x", torch.float32, (2, 8), None), (-1, x, "x", torch.float32, (2, 8), None), (0, x)):
        with pytest.raises(TypeError):
            on_device(*args)
    assert on_device(0, None, "x", torch.float32, (2, 8), None) is None


def test_reference_by_hand():
    codes, e = quantise64(torch.tensor([[448.0, 1.0, -0.3], [449.0, 1.0, 27.0], [0.0, 0.0, 0.0], [1.0, math.inf, math.nan]]))
    assert e.tolist() == [0, 1, -117, -8]
    assert codes[0].tolist() == [448.0, 1.0, -0.3125] and codes[1].tolist() == [224.0, 0.5, 14.0]
    assert codes[2].tolist() == [0.0, 0.0, 0.0] and codes[3, 0] == 256 and torch.isnan(codes[3, 1:]).all()
    x = torch.randn(500, 40, generator=torch.Generator().manual_seed(0)) * 10.0
    codes, e = quantise64(x)
    assert torch.equal(codes, torch.ldexp(x, -e[:, None]).to(E4M3).double())
    assert (codes.abs().amax(1) <= 448).all() and (codes.abs().amax(1) >= 208).all()
    s = lambda *a: seen64(*a).int().tolist()  # noqa: E731
    assert s(2, 3, 0, 0) == [[1, 1, 0], [1, 1, 1]] and s(3, 2, 0, 0) == [[0, 0], [1, 0], [1, 1]]
    assert s(1, 5, 2, 1) == [[1, 0, 0, 1, 1]] and s(2, 4, 1, 3) == [[1, 1, 1, 0], [1, 1, 1, 1]]


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("batch", [8, 64, 128, 256, 500, 1024])
def test_single_tokens_of_any_batch_are_divided(batch, cache):
    """A long sequence among many short ones has to be cut, or one workgroup reads it alone: such calls have a workspace."""
    m = cc()
    d = m.paged_attention_desc_create(m.make_paged_attention_params(32, 8, 128, 16, dtype="bf16", cache_dtype=cache))
    assert m.paged_attention_workspace_bytes(d, batch, batch, 8192) > 0


def _kv(heads, d, ps, **kw):
    m = cc()
    return m.kv_cache_desc_create(m.make_kv_cache_params(heads, d, ps, dtype="bf16", cache_dtype="e4m3", **kw))


# (strides of keys and values, of the scales, where values and the two scales begin behind the keys) of pages of 8
# tokens, 4 heads of 64 codes.
INTERLEAVED = {
    "keys and values a token": ((4096, 512, 64), None, (256, P, 2 * P)),
    "keys and values a head": ((4096, 512, 128), None, (64, P, 2 * P)),
    "heads outermost": ((512, 64, 1 << 20), None, (1 << 19, P, 2 * P)),
    "scales behind their rows": ((2560, 320, 80), (2560, 320, 80), (P, 64, P + 64)),
    "all of a head together": ((5120, 640, 160), (5120, 640, 160), (80, 64, 144)),
}


@pytest.mark.parametrize("name", INTERLEAVED)
def test_interleaved_pages_do_not_overlap(name):
    """Rows in each other's gaps are no overlap; a row that reaches one byte into another is.  The last check, of the
    values' scales against the slots, refuses each call before any launch."""
    m = cc()
    strides, scales, (dv, dks, dvs) = INTERLEAVED[name]
    desc = _kv(4, 64, 8, k_page_strides=strides, v_page_strides=strides, scale_strides=scales)
    k, v, base = 8 * P, 9 * P, P
    slots = base + dvs + (7 * scales[1] + 3 * scales[2] if scales else 0)   # where the values' scales alone end

    def status(dv=dv, dks=dks, dvs=dvs):
        return (m._lib.kv_cache_store(desc.handle, 4, k, v, slots, 60, base, base + dv, base + dks, base + dvs, None),
                m.conv2d_last_error())
    assert status() == (m.CONV_ERR_ALIAS, "pages or scales overlap an input")
    for at in (63,) if scales else (63, -63, strides[0] * 59 + strides[1] * 7 + strides[2] * 3 + 63):
        assert status(dv=at) == (m.CONV_ERR_ALIAS, "pages or scales overlap each other"), at
    if scales:
        for change in (dict(dks=63), dict(dks=0), dict(dks=scales[0] * 5 + scales[1] * 3 + 1)):
            assert status(**change) == (m.CONV_ERR_ALIAS, "pages or scales overlap each other"), change


def test_interleaved_rows_of_a_load_do_not_overlap():
    """Keys and values in token rows of one buffer, sequences padded; refused for the table, which overlaps the values."""
    m = cc()
    desc = _kv(4, 64, 8, k_stride=512, v_stride=512, k_batch_stride=512 * 100, v_batch_stride=512 * 100)
    k, table = 8 * P, 8 * P + 512
    status = lambda v: (m._lib.kv_cache_load(desc.handle, 3, 90, 12, table, None, 60, P, 2 * P, 3 * P, 4 * P, k, v, None),  # noqa: E731
                        m.conv2d_last_error())
    assert status(k + 512) == (m.CONV_ERR_ALIAS, "k or v overlaps page_table or kv_lens")
    assert status(k + 510) == (m.CONV_ERR_ALIAS, "k overlaps v") and status(k + 2 * 51200 * 2) == (m.CONV_ERR_ALIAS, "k overlaps v")
