"""Python binding of include/attention.h: linear, qk_rope and attention.

Argument marshalling only, as for the convolutions: torch tensors give device
memory and the current stream, the binding checks device, type, shape and
strides against the descriptor (_marshal, csrc/marshal.cpp: compiled, since the
checks in Python cost as much as the launch), and passes raw pointers through
the C ABI.
Sizes that a call may change (rows, tokens, batch and lengths) come from the
tensors' shapes.

    d = linear_desc_create(make_linear_params(k, n, act="gelu", has_bias=True, dtype="bf16"))
    linear_forward(d, x, w, bias, None, y)
"""
import ctypes

from . import (CONV_OK, ConvError, DTYPE_F32, _ACT_NAMES, _DTYPE_NAMES, _lib, _stream, conv2d_last_error)

LINEAR_ACT_SILU, LINEAR_ACT_GELU, LINEAR_ACT_GELU_TANH = 16, 17, 18
ROPE_HALF, ROPE_INTERLEAVED = range(2)
ROPE_SCALING_NONE, ROPE_SCALING_LINEAR, ROPE_SCALING_YARN = range(3)

_LINEAR_ACTS = dict(_ACT_NAMES, silu=LINEAR_ACT_SILU, gelu=LINEAR_ACT_GELU, gelu_tanh=LINEAR_ACT_GELU_TANH)
_LAYOUTS = {"half": ROPE_HALF, "interleaved": ROPE_INTERLEAVED}
_SCALINGS = {"none": ROPE_SCALING_NONE, "linear": ROPE_SCALING_LINEAR, "yarn": ROPE_SCALING_YARN}


def _fields(kind, names):
    return [(n, kind) for n in names.split()]


class linear_params_t(ctypes.Structure):
    _fields_ = (_fields(ctypes.c_int64, "x_stride y_stride residual_stride") +
                _fields(ctypes.c_int32, "k n has_bias has_residual act_type") +
                [("act_params", ctypes.c_float * 2), ("dtype", ctypes.c_int32)])


class qk_rope_params_t(ctypes.Structure):
    _fields_ = (_fields(ctypes.c_int64, "qkv_stride q_stride k_stride v_stride") +
                _fields(ctypes.c_double, "theta factor beta_fast beta_slow attn_factor") +
                _fields(ctypes.c_int32, "heads_q heads_kv head_dim rotary_dim layout scaling original_len has_norm") +
                [("eps", ctypes.c_float), ("dtype", ctypes.c_int32)])


class attention_params_t(ctypes.Structure):
    _fields_ = (_fields(ctypes.c_int64 * 3, "q_strides k_strides v_strides out_strides") +
                _fields(ctypes.c_int32, "heads_q heads_kv head_dim causal window has_slopes") +
                _fields(ctypes.c_float, "softcap scale") + [("dtype", ctypes.c_int32)])


# C ABI symbols of include/attention.h.
EXPORTED = ("linear_params_init", "linear_desc_create", "linear_desc_destroy", "linear_desc_kernel_name",
            "linear_forward", "qk_rope_params_init", "qk_rope_desc_create", "qk_rope_desc_destroy", "qk_rope_forward",
            "attention_params_init", "attention_desc_create", "attention_desc_destroy", "attention_workspace_bytes",
            "attention_forward")


def _declare():
    vp, i32, i64, P = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.POINTER
    for name, params in (("linear", linear_params_t), ("qk_rope", qk_rope_params_t),
                         ("attention", attention_params_t)):
        init, create = getattr(_lib, name + "_params_init"), getattr(_lib, name + "_desc_create")
        init.argtypes, init.restype = [P(params)], None
        create.argtypes, create.restype = [P(params), P(vp)], i32
        destroy = getattr(_lib, name + "_desc_destroy")
        destroy.argtypes, destroy.restype = [vp], None
    _lib.linear_desc_kernel_name.argtypes, _lib.linear_desc_kernel_name.restype = [vp, i64], ctypes.c_char_p
    _lib.linear_forward.argtypes, _lib.linear_forward.restype = [vp, i64] + [vp] * 6, i32
    _lib.qk_rope_forward.argtypes = [vp, i64] + [vp] * 5 + [i64] + [vp] * 4
    _lib.qk_rope_forward.restype = i32
    _lib.attention_workspace_bytes.argtypes, _lib.attention_workspace_bytes.restype = [vp, i64, i64, i64, P(i64)], i32
    _lib.attention_forward.argtypes = [vp, i64, i64, i64] + [vp] * 7 + [i32] + [vp] * 3 + [i64, vp]
    _lib.attention_forward.restype = i32


_declare()


def _check(status):
    if status != CONV_OK:
        raise ConvError(status, conv2d_last_error())


class _Desc:
    """Owns a descriptor of include/attention.h; destroyed with the object."""

    def __init__(self, kind, params):
        if _tensor is None:
            _load()
        h = ctypes.c_void_p()
        _check(getattr(_lib, kind + "_desc_create")(ctypes.byref(params), ctypes.byref(h)))
        self.kind, self.handle = kind, h
        self.params = type(params)()
        ctypes.memmove(ctypes.byref(self.params), ctypes.byref(params), ctypes.sizeof(params))
        self.dtype = _f32 if params.dtype == DTYPE_F32 else _bf16
        # Kept on the instance: module globals may already be gone when the
        # last descriptors are collected at interpreter exit.
        self._destroy = getattr(_lib, kind + "_desc_destroy")

    def __del__(self):
        self.close()

    def close(self):
        if getattr(self, "handle", None) and getattr(self, "_destroy", None) is not None:
            self._destroy(self.handle)
            self.handle = None


def _init(params, name):
    p = params()
    getattr(_lib, name)(ctypes.byref(p))
    return p


def _code(v, names):
    return int(names[v] if isinstance(v, str) else v)


_tensor = None    # _marshal.tensor: the device pointer of a GPU tensor of a type, shape and strides (None: dense)
_f32 = _bf16 = _i32 = None


def _load():
    """Types and the compiled checks of tensors, which need torch: at the first descriptor."""
    global _tensor, _f32, _bf16, _i32
    import torch

    try:
        from ._marshal import tensor
    except ImportError as e:
        raise ImportError(f"the binding's tensor checks (_marshal.so) are not built, build.py makes them: {e}") from e
    _tensor, _f32, _bf16, _i32 = tensor, torch.float32, torch.bfloat16, torch.int32


# -------------------------------------------------------------- linear --

def linear_params_init() -> linear_params_t:
    return _init(linear_params_t, "linear_params_init")


def make_linear_params(k, n, *, has_bias=False, act="none", alpha=None, clip=None, has_residual=False, x_stride=0,
                       y_stride=0, residual_stride=0, dtype="f32") -> linear_params_t:
    """Keyword construction; act: a name ("none", "relu", "leaky_relu", "clip",
    "silu", "gelu", "gelu_tanh") or a code."""
    p = linear_params_init()
    p.k, p.n, p.has_bias, p.has_residual = int(k), int(n), int(bool(has_bias)), int(bool(has_residual))
    p.x_stride, p.y_stride, p.residual_stride = int(x_stride), int(y_stride), int(residual_stride)
    p.act_type = _code(act, _LINEAR_ACTS)
    if alpha is not None:
        p.act_params[0] = float(alpha)
    if clip is not None:
        p.act_params[0], p.act_params[1] = float(clip[0]), float(clip[1])
    p.dtype = _code(dtype, _DTYPE_NAMES)
    return p


def linear_desc_create(params: linear_params_t) -> _Desc:
    d = _Desc("linear", params)
    p = d.params
    d.x_strides, d.y_strides = (p.x_stride or p.k, 1), (p.y_stride or p.n, 1)
    d.r_strides = (p.residual_stride or p.n, 1)
    d.k, d.n, d.w_shape, d.w_strides, d.b_shape = p.k, p.n, (p.n, p.k), (p.k, 1), (p.n,)
    d.has_bias, d.has_residual = bool(p.has_bias), bool(p.has_residual)
    return d


def linear_desc_destroy(desc: _Desc) -> None:
    desc.close()


def linear_desc_kernel_name(desc: _Desc, rows: int) -> str:
    return _lib.linear_desc_kernel_name(desc.handle, int(rows)).decode()


def linear_forward(desc: _Desc, x, w, bias, residual, y, stream=None) -> None:
    """y = act(x w^T + bias) + residual; x [rows, k], w [n, k], bias float32 [n],
    residual and y [rows, n] (y may be the residual itself)."""
    dt, rows = desc.dtype, x.shape[0]
    y_shape = (rows, desc.n)
    _check(_lib.linear_forward(
        desc.handle, rows, _tensor(x, "x", dt, (rows, desc.k), desc.x_strides),
        _tensor(w, "w", dt, desc.w_shape, desc.w_strides),
        _tensor(bias, "bias", _f32, desc.b_shape, None) if desc.has_bias else None,
        _tensor(residual, "residual", dt, y_shape, desc.r_strides) if desc.has_residual else None,
        _tensor(y, "y", dt, y_shape, desc.y_strides), _stream(stream)))


# ------------------------------------------------------------- qk_rope --

def qk_rope_params_init() -> qk_rope_params_t:
    return _init(qk_rope_params_t, "qk_rope_params_init")


def make_qk_rope_params(heads_q, heads_kv, head_dim, *, rotary_dim=0, layout="half", has_norm=False, eps=1e-6,
                        theta=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0,
                        attn_factor=0.0, qkv_stride=0, q_stride=0, k_stride=0, v_stride=0,
                        dtype="f32") -> qk_rope_params_t:
    p = qk_rope_params_init()
    p.heads_q, p.heads_kv, p.head_dim, p.rotary_dim = int(heads_q), int(heads_kv), int(head_dim), int(rotary_dim)
    p.layout, p.scaling = _code(layout, _LAYOUTS), _code(scaling, _SCALINGS)
    p.has_norm, p.eps, p.theta, p.factor = int(bool(has_norm)), float(eps), float(theta), float(factor)
    p.original_len, p.beta_fast, p.beta_slow = int(original_len), float(beta_fast), float(beta_slow)
    p.attn_factor = float(attn_factor)
    p.qkv_stride, p.q_stride, p.k_stride, p.v_stride = int(qkv_stride), int(q_stride), int(k_stride), int(v_stride)
    p.dtype = _code(dtype, _DTYPE_NAMES)
    return p


def qk_rope_desc_create(params: qk_rope_params_t) -> _Desc:
    d = _Desc("qk_rope", params)
    p = d.params
    d.width = (p.heads_q + 2 * p.heads_kv) * p.head_dim
    d.qkv_strides = (p.qkv_stride or d.width, 1)
    d.q_strides = (p.q_stride or p.heads_q * p.head_dim, p.head_dim, 1)
    d.k_strides = (p.k_stride or p.heads_kv * p.head_dim, p.head_dim, 1)
    d.v_strides = (p.v_stride or p.heads_kv * p.head_dim, p.head_dim, 1)
    d.heads_q, d.heads_kv, d.head_dim, d.g_shape, d.has_norm = (p.heads_q, p.heads_kv, p.head_dim, (p.head_dim,),
                                                                bool(p.has_norm))
    return d


def qk_rope_desc_destroy(desc: _Desc) -> None:
    desc.close()


def qk_rope_forward(desc: _Desc, qkv, q_gamma, k_gamma, positions, slots, q, k, v, stream=None) -> None:
    """Norm and rotation of qkv [tokens, (heads_q + 2 heads_kv) head_dim]:
    queries to q [tokens, heads_q, head_dim], keys and values to rows `slots`
    (None: the token's own number) of k and v [cache_rows, heads_kv, head_dim].
    positions and slots are int32; v None: values are not stored."""
    dt, tokens, rows = desc.dtype, qkv.shape[0], k.shape[0]
    token_shape, kv_shape = (tokens,), (rows, desc.heads_kv, desc.head_dim)
    _check(_lib.qk_rope_forward(
        desc.handle, tokens, _tensor(qkv, "qkv", dt, (tokens, desc.width), desc.qkv_strides),
        _tensor(q_gamma, "q_gamma", _f32, desc.g_shape, None) if desc.has_norm else None,
        _tensor(k_gamma, "k_gamma", _f32, desc.g_shape, None) if desc.has_norm else None,
        _tensor(positions, "positions", _i32, token_shape, None), _tensor(slots, "slots", _i32, token_shape, None), rows,
        _tensor(q, "q", dt, (tokens, desc.heads_q, desc.head_dim), desc.q_strides),
        _tensor(k, "k", dt, kv_shape, desc.k_strides), _tensor(v, "v", dt, kv_shape, desc.v_strides), _stream(stream)))


# ----------------------------------------------------------- attention --

def attention_params_init() -> attention_params_t:
    return _init(attention_params_t, "attention_params_init")


def make_attention_params(heads_q, heads_kv, head_dim, *, q_strides, k_strides, v_strides, out_strides, causal=False,
                          window=0, softcap=0.0, has_slopes=False, scale=None, dtype="f32") -> attention_params_t:
    """Strides: (batch, token, head) of each tensor, in elements."""
    p = attention_params_init()
    p.heads_q, p.heads_kv, p.head_dim = int(heads_q), int(heads_kv), int(head_dim)
    for field, s in (("q_strides", q_strides), ("k_strides", k_strides), ("v_strides", v_strides),
                     ("out_strides", out_strides)):
        setattr(p, field, (ctypes.c_int64 * 3)(*(int(v) for v in s)))
    p.causal, p.window, p.has_slopes = int(bool(causal)), int(window), int(bool(has_slopes))
    p.softcap = float(softcap)
    if scale is not None:
        p.scale = float(scale)
    p.dtype = _code(dtype, _DTYPE_NAMES)
    return p


def attention_desc_create(params: attention_params_t) -> _Desc:
    d = _Desc("attention", params)
    p = d.params
    d.strides = [tuple(s) + (1,) for s in (p.q_strides, p.k_strides, p.v_strides, p.out_strides)]
    d.heads_q, d.heads_kv, d.head_dim, d.has_slopes = p.heads_q, p.heads_kv, p.head_dim, bool(p.has_slopes)
    return d


def attention_desc_destroy(desc: _Desc) -> None:
    desc.close()


def attention_workspace_bytes(desc: _Desc, batch: int, q_len: int, kv_len: int) -> int:
    n = ctypes.c_int64()
    _check(_lib.attention_workspace_bytes(desc.handle, int(batch), int(q_len), int(kv_len), ctypes.byref(n)))
    return n.value


def attention_forward(desc: _Desc, q, k, v, out, *, q_lens=None, kv_lens=None, prefix_lens=None, doc_offsets=None,
                      slopes=None, workspace=None, stream=None) -> None:
    """Attention of q [batch, q_len, heads_q, head_dim] over k, v [batch, kv_len,
    heads_kv, head_dim] into out (q's shape).  q_lens, kv_lens, prefix_lens:
    int32 [batch]; doc_offsets: int32 [batch, documents + 1]; slopes: float32
    [heads_q]; workspace: a tensor of attention_workspace_bytes, or None where
    that is 0."""
    dt, hd = desc.dtype, desc.head_dim
    (batch, q_len), kv_len = q.shape[:2], k.shape[1]
    q_shape, k_shape, b_shape = (batch, q_len, desc.heads_q, hd), (batch, kv_len, desc.heads_kv, hd), (batch,)
    sq, sk, sv, so = desc.strides
    n_docs, ws, ws_bytes = 0, None, 0
    if doc_offsets is not None:
        n_docs = doc_offsets.shape[-1] - 1
    if workspace is not None:
        if not (workspace.is_cuda and workspace.is_contiguous()):
            raise ValueError("workspace: contiguous GPU tensor expected")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(_lib.attention_forward(
        desc.handle, batch, q_len, kv_len, _tensor(q, "q", dt, q_shape, sq), _tensor(k, "k", dt, k_shape, sk),
        _tensor(v, "v", dt, k_shape, sv), _tensor(q_lens, "q_lens", _i32, b_shape, None),
        _tensor(kv_lens, "kv_lens", _i32, b_shape, None), _tensor(prefix_lens, "prefix_lens", _i32, b_shape, None),
        _tensor(doc_offsets, "doc_offsets", _i32, (batch, n_docs + 1), None), n_docs,
        _tensor(slopes, "slopes", _f32, (desc.heads_q,), None) if desc.has_slopes else None,
        _tensor(out, "out", dt, q_shape, so), ws, ws_bytes, _stream(stream)))
