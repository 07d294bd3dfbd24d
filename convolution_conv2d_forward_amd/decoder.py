"""Python binding of include/decoder.h: kv_cache, paged_attention and block_norm.

Argument marshalling only, as in attention.py: torch tensors give device memory
and the current stream, compiled checks (_marshal) hold device, type, shape and
strides against the descriptor, and raw pointers go through the C ABI.  Sizes
that a call may change (tokens, batch, rows, pages) come from the tensors'
shapes.  All tensors of a call lie on the current device, and so does the stream:
a torch stream of another device is refused; of a raw handle it is not known.

    d = kv_cache_desc_create(make_kv_cache_params(8, 128, 16, dtype="bf16", cache_dtype="e4m3"))
    kv_cache_store(d, k, v, slots, k_pages, v_pages, k_scales, v_scales)
"""
import ctypes

from . import DTYPE_F32, _DTYPE_NAMES, _lib, _stream, _torch
from .attention import _check, _code, _Desc, _fields, _init

KV_CACHE_E4M3 = 16
BLOCK_NORM_NONE, BLOCK_NORM_RMS, BLOCK_NORM_LAYER = range(3)

_CACHES = dict(_DTYPE_NAMES, e4m3=KV_CACHE_E4M3)
_NORMS = {"none": BLOCK_NORM_NONE, "rms": BLOCK_NORM_RMS, "layer": BLOCK_NORM_LAYER}


class kv_cache_params_t(ctypes.Structure):
    _fields_ = (_fields(ctypes.c_int64, "k_stride v_stride k_batch_stride v_batch_stride") +
                _fields(ctypes.c_int64 * 3, "k_page_strides v_page_strides scale_strides") +
                _fields(ctypes.c_int32, "heads_kv head_dim page_size dtype cache_dtype"))


class paged_attention_params_t(ctypes.Structure):
    _fields_ = (_fields(ctypes.c_int64, "q_stride out_stride") +
                _fields(ctypes.c_int64 * 3, "k_page_strides v_page_strides scale_strides") +
                _fields(ctypes.c_int32, "heads_q heads_kv head_dim page_size window sinks") +
                _fields(ctypes.c_float, "softcap scale") + _fields(ctypes.c_int32, "dtype cache_dtype"))


class block_norm_params_t(ctypes.Structure):
    _fields_ = (_fields(ctypes.c_int64, "y_stride x_stride residual_stride out_stride gate_stride") +
                _fields(ctypes.c_int32, "width post_norm pre_norm has_post_beta has_pre_beta has_gate gate_rows") +
                _fields(ctypes.c_float, "residual_scale block_scale eps") + [("dtype", ctypes.c_int32)])


# C ABI symbols of include/decoder.h.
EXPORTED = ("kv_cache_params_init", "kv_cache_desc_create", "kv_cache_desc_destroy", "kv_cache_store",
            "kv_cache_load", "paged_attention_params_init", "paged_attention_desc_create",
            "paged_attention_desc_destroy", "paged_attention_workspace_bytes", "paged_attention_forward",
            "block_norm_params_init", "block_norm_desc_create", "block_norm_desc_destroy", "block_norm_forward")


def _declare():
    vp, i32, i64, P = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.POINTER
    for name, params in (("kv_cache", kv_cache_params_t), ("paged_attention", paged_attention_params_t),
                         ("block_norm", block_norm_params_t)):
        init, create = getattr(_lib, name + "_params_init"), getattr(_lib, name + "_desc_create")
        init.argtypes, init.restype = [P(params)], None
        create.argtypes, create.restype = [P(params), P(vp)], i32
        destroy = getattr(_lib, name + "_desc_destroy")
        destroy.argtypes, destroy.restype = [vp], None
    _lib.kv_cache_store.argtypes, _lib.kv_cache_store.restype = [vp, i64] + [vp] * 3 + [i64] + [vp] * 5, i32
    _lib.kv_cache_load.argtypes = [vp, i64, i64, i64, vp, vp, i64] + [vp] * 7
    _lib.kv_cache_load.restype = i32
    _lib.paged_attention_workspace_bytes.argtypes = [vp, i64, i64, i64, P(i64)]
    _lib.paged_attention_workspace_bytes.restype = i32
    _lib.paged_attention_forward.argtypes = [vp, i64, i64, i64] + [vp] * 4 + [i64] + [vp] * 6 + [i64, vp]
    _lib.paged_attention_forward.restype = i32
    _lib.block_norm_forward.argtypes, _lib.block_norm_forward.restype = [vp, i64] + [vp] * 10, i32


_declare()

_tensor = None   # _marshal.on_device
_f32 = _bf16 = _i32 = _u8 = _e4m3 = _device = None


def _load():
    """Types and the compiled checks of tensors: at the first descriptor."""
    global _tensor, _f32, _bf16, _i32, _u8, _e4m3, _device
    torch = _torch()
    from ._marshal import on_device
    _f32, _bf16, _i32, _u8, _e4m3 = torch.float32, torch.bfloat16, torch.int32, torch.uint8, torch.float8_e4m3fn
    _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _tensor = on_device


def _desc(kind, params):
    d = _Desc(kind, params)
    if _tensor is None:
        _load()
    return d


def _on(stream):
    """Number of the device that a call with this stream runs on."""
    index = getattr(stream, "device_index", None)
    here = _device()
    if index is not None and index != here:
        raise ValueError(f"the stream is on cuda:{index}, the current device is cuda:{here}")
    return here


def _strides(p, field, value):
    if value is not None:
        setattr(p, field, (ctypes.c_int64 * 3)(*(int(v) for v in value)))


def _page_strides(s, page_size, heads, width):
    """The descriptor's (page, token, head) strides, all 0 standing for dense ones, and an element's."""
    s = tuple(s)
    if s == (0, 0, 0):
        s = (page_size * heads * width, heads * width, width)
    return s


def _workspace(workspace, device):
    if workspace is None:
        return None, 0
    if not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace: contiguous GPU tensor expected")
    if workspace.get_device() != device:
        raise ValueError(f"workspace: on cuda:{workspace.get_device()}, the call runs on cuda:{device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


class _Cache:
    """What the pages of a descriptor's cache look like."""

    def __init__(self, p):
        self.quantised = p.cache_dtype == KV_CACHE_E4M3
        self.dtype = _e4m3 if self.quantised else _f32 if p.cache_dtype == DTYPE_F32 else _bf16
        self.inner = (p.page_size, p.heads_kv, p.head_dim)
        self.k = _page_strides(p.k_page_strides, p.page_size, p.heads_kv, p.head_dim) + (1,)
        self.v = _page_strides(p.v_page_strides, p.page_size, p.heads_kv, p.head_dim) + (1,)
        self.scales = _page_strides(p.scale_strides, p.page_size, p.heads_kv, 1)

    def pointers(self, dev, k_pages, v_pages, k_scales, v_scales):
        n = k_pages.shape[0]
        shape = (n,) + self.inner
        got = (n, _tensor(dev, k_pages, "k_pages", self.dtype, shape, self.k),
               _tensor(dev, v_pages, "v_pages", self.dtype, shape, self.v))
        if not self.quantised:
            return got + (None, None)
        shape = shape[:3]
        return got + (_tensor(dev, k_scales, "k_scales", _u8, shape, self.scales),
                      _tensor(dev, v_scales, "v_scales", _u8, shape, self.scales))


# ------------------------------------------------------------ kv_cache --

def kv_cache_params_init() -> kv_cache_params_t:
    return _init(kv_cache_params_t, "kv_cache_params_init")


def make_kv_cache_params(heads_kv, head_dim, page_size, *, dtype="f32", cache_dtype=None, k_stride=0, v_stride=0,
                         k_batch_stride=0, v_batch_stride=0, k_page_strides=None, v_page_strides=None,
                         scale_strides=None) -> kv_cache_params_t:
    """cache_dtype: "e4m3", or dtype's own (None).  Page strides: (page, token, head), in elements; None: dense."""
    p = kv_cache_params_init()
    p.heads_kv, p.head_dim, p.page_size = int(heads_kv), int(head_dim), int(page_size)
    p.k_stride, p.v_stride = int(k_stride), int(v_stride)
    p.k_batch_stride, p.v_batch_stride = int(k_batch_stride), int(v_batch_stride)
    for field, s in (("k_page_strides", k_page_strides), ("v_page_strides", v_page_strides),
                     ("scale_strides", scale_strides)):
        _strides(p, field, s)
    p.dtype = _code(dtype, _DTYPE_NAMES)
    p.cache_dtype = p.dtype if cache_dtype is None else _code(cache_dtype, _CACHES)
    return p


def kv_cache_desc_create(params: kv_cache_params_t) -> _Desc:
    d = _desc("kv_cache", params)
    p = d.params
    d.cache, d.heads, d.head_dim = _Cache(p), p.heads_kv, p.head_dim
    row = p.heads_kv * p.head_dim
    d.k_stride, d.v_stride = p.k_stride or row, p.v_stride or row
    d.k_strides, d.v_strides = (d.k_stride, p.head_dim, 1), (d.v_stride, p.head_dim, 1)
    return d


def kv_cache_desc_destroy(desc: _Desc) -> None:
    desc.close()


def kv_cache_store(desc: _Desc, k, v, slots, k_pages, v_pages, k_scales=None, v_scales=None, stream=None) -> None:
    """Stores k, v [tokens, heads_kv, head_dim] to the int32 slots [tokens] of the pages [n_pages, page_size, heads_kv,
    head_dim]; an E4M3 cache (torch.float8_e4m3fn) has scales, uint8 [n_pages, page_size, heads_kv]."""
    dev, dt = _on(stream), desc.dtype
    shape = (k.shape[0], desc.heads, desc.head_dim)
    _check(_lib.kv_cache_store(
        desc.handle, shape[0], _tensor(dev, k, "k", dt, shape, desc.k_strides),
        _tensor(dev, v, "v", dt, shape, desc.v_strides), _tensor(dev, slots, "slots", _i32, shape[:1], None),
        *desc.cache.pointers(dev, k_pages, v_pages, k_scales, v_scales), _stream(stream)))


def kv_cache_load(desc: _Desc, page_table, kv_lens, k_pages, v_pages, k_scales, v_scales, k, v, stream=None) -> None:
    """Reads the first kv_lens (int32 [batch]; None: all) tokens of each sequence from the pages that page_table (int32
    [batch, max_pages]) lists, into rows of k and v [batch, kv_len, heads_kv, head_dim]; other rows stay."""
    dev, dt, p = _on(stream), desc.dtype, desc.params
    (batch, max_pages), kv_len = page_table.shape, k.shape[1]
    shape = (batch, kv_len, desc.heads, desc.head_dim)
    n, kp, vp, ks, vs = desc.cache.pointers(dev, k_pages, v_pages, k_scales, v_scales)
    _check(_lib.kv_cache_load(
        desc.handle, batch, kv_len, max_pages, _tensor(dev, page_table, "page_table", _i32, (batch, max_pages), None),
        _tensor(dev, kv_lens, "kv_lens", _i32, (batch,), None), n, kp, vp, ks, vs,
        _tensor(dev, k, "k", dt, shape, (p.k_batch_stride or kv_len * desc.k_stride,) + desc.k_strides),
        _tensor(dev, v, "v", dt, shape, (p.v_batch_stride or kv_len * desc.v_stride,) + desc.v_strides),
        _stream(stream)))


# ----------------------------------------------------- paged_attention --

def paged_attention_params_init() -> paged_attention_params_t:
    return _init(paged_attention_params_t, "paged_attention_params_init")


def make_paged_attention_params(heads_q, heads_kv, head_dim, page_size, *, window=0, sinks=0, softcap=0.0, scale=None,
                                dtype="f32", cache_dtype=None, q_stride=0, out_stride=0, k_page_strides=None,
                                v_page_strides=None, scale_strides=None) -> paged_attention_params_t:
    """cache_dtype: "e4m3", or dtype's own (None).  Page strides: (page, token, head), in elements; None: dense."""
    p = paged_attention_params_init()
    p.heads_q, p.heads_kv, p.head_dim, p.page_size = int(heads_q), int(heads_kv), int(head_dim), int(page_size)
    p.window, p.sinks, p.softcap = int(window), int(sinks), float(softcap)
    if scale is not None:
        p.scale = float(scale)
    p.q_stride, p.out_stride = int(q_stride), int(out_stride)
    for field, s in (("k_page_strides", k_page_strides), ("v_page_strides", v_page_strides),
                     ("scale_strides", scale_strides)):
        _strides(p, field, s)
    p.dtype = _code(dtype, _DTYPE_NAMES)
    p.cache_dtype = p.dtype if cache_dtype is None else _code(cache_dtype, _CACHES)
    return p


def paged_attention_desc_create(params: paged_attention_params_t) -> _Desc:
    d = _desc("paged_attention", params)
    p = d.params
    d.cache, d.row = _Cache(p), (p.heads_q, p.head_dim)
    d.q_strides = (p.q_stride or p.heads_q * p.head_dim, p.head_dim, 1)
    d.out_strides = (p.out_stride or p.heads_q * p.head_dim, p.head_dim, 1)
    return d


def paged_attention_desc_destroy(desc: _Desc) -> None:
    desc.close()


def paged_attention_workspace_bytes(desc: _Desc, tokens: int, batch: int, max_pages: int) -> int:
    n = ctypes.c_int64()
    _check(_lib.paged_attention_workspace_bytes(desc.handle, int(tokens), int(batch), int(max_pages), ctypes.byref(n)))
    return n.value


def paged_attention_forward(desc: _Desc, q, q_offsets, kv_lens, page_table, k_pages, v_pages, k_scales, v_scales, out,
                            *, workspace=None, stream=None) -> None:
    """Attention of the new tokens q [tokens, heads_q, head_dim], sequence b's being rows q_offsets[b] ..
    q_offsets[b + 1] - 1 (int32 [batch + 1]), over their kv_lens (int32 [batch]) cached tokens, on the pages that
    page_table (int32 [batch, max_pages]) lists, into out (q's shape).  The scales are None unless the cache is E4M3;
    workspace: a tensor of paged_attention_workspace_bytes, or None where that is 0."""
    dev, dt = _on(stream), desc.dtype
    tokens, (batch, max_pages) = q.shape[0], page_table.shape
    shape = (tokens,) + desc.row
    _check(_lib.paged_attention_forward(
        desc.handle, tokens, batch, max_pages, _tensor(dev, q, "q", dt, shape, desc.q_strides),
        _tensor(dev, q_offsets, "q_offsets", _i32, (batch + 1,), None),
        _tensor(dev, kv_lens, "kv_lens", _i32, (batch,), None),
        _tensor(dev, page_table, "page_table", _i32, (batch, max_pages), None),
        *desc.cache.pointers(dev, k_pages, v_pages, k_scales, v_scales),
        _tensor(dev, out, "out", dt, shape, desc.out_strides), *_workspace(workspace, dev), _stream(stream)))


# ---------------------------------------------------------- block_norm --

def block_norm_params_init() -> block_norm_params_t:
    return _init(block_norm_params_t, "block_norm_params_init")


def make_block_norm_params(width, *, post_norm="none", pre_norm="none", has_post_beta=False, has_pre_beta=False,
                           has_gate=False, gate_rows=0, residual_scale=1.0, block_scale=1.0, eps=1e-6, y_stride=0,
                           x_stride=0, residual_stride=0, out_stride=0, gate_stride=0,
                           dtype="f32") -> block_norm_params_t:
    """Norms: "none", "rms", "layer" or a code."""
    p = block_norm_params_init()
    p.width, p.post_norm, p.pre_norm = int(width), _code(post_norm, _NORMS), _code(pre_norm, _NORMS)
    p.has_post_beta, p.has_pre_beta, p.has_gate = int(bool(has_post_beta)), int(bool(has_pre_beta)), int(bool(has_gate))
    p.gate_rows, p.residual_scale, p.block_scale = int(gate_rows), float(residual_scale), float(block_scale)
    p.eps, p.y_stride, p.x_stride, p.residual_stride = float(eps), int(y_stride), int(x_stride), int(residual_stride)
    p.out_stride, p.gate_stride = int(out_stride), int(gate_stride)
    p.dtype = _code(dtype, _DTYPE_NAMES)
    return p


def block_norm_desc_create(params: block_norm_params_t) -> _Desc:
    d = _desc("block_norm", params)
    p = d.params
    d.width, d.vector, d.gate_rows = p.width, (p.width,), p.gate_rows
    d.strides = [(getattr(p, n + "_stride") or p.width, 1) for n in ("y", "x", "residual", "out", "gate")]
    d.post, d.pre = p.post_norm != BLOCK_NORM_NONE, p.pre_norm != BLOCK_NORM_NONE
    d.has_gate, d.post_beta, d.pre_beta = bool(p.has_gate), bool(p.has_post_beta), bool(p.has_pre_beta)
    return d


def block_norm_desc_destroy(desc: _Desc) -> None:
    desc.close()


def block_norm_forward(desc: _Desc, y, x, gate, post_gamma, post_beta, pre_gamma, pre_beta, residual, out,
                       stream=None) -> None:
    """residual = residual_scale * x + block_scale * gate * post(y), out = pre(residual): y, x, residual and out [rows,
    width], gate [ceil(rows / gate_rows), width] ([1, width] for gate_rows = 0), gammas and betas float32 [width]; what
    the descriptor has not is None.  residual may be x or y itself, out may be y."""
    dev, dt, rows, vector = _on(stream), desc.dtype, y.shape[0], desc.vector
    shape, (sy, sx, sr, so, sg) = (rows, desc.width), desc.strides
    gates = (-(-rows // desc.gate_rows) if desc.gate_rows else 1, desc.width)
    _check(_lib.block_norm_forward(
        desc.handle, rows, _tensor(dev, y, "y", dt, shape, sy), _tensor(dev, x, "x", dt, shape, sx),
        _tensor(dev, gate, "gate", dt, gates, sg) if desc.has_gate else None,
        _tensor(dev, post_gamma, "post_gamma", _f32, vector, None) if desc.post else None,
        _tensor(dev, post_beta, "post_beta", _f32, vector, None) if desc.post_beta else None,
        _tensor(dev, pre_gamma, "pre_gamma", _f32, vector, None) if desc.pre else None,
        _tensor(dev, pre_beta, "pre_beta", _f32, vector, None) if desc.pre_beta else None,
        _tensor(dev, residual, "residual", dt, shape, sr),
        _tensor(dev, out, "out", dt, shape, so) if desc.pre else None, _stream(stream)))
