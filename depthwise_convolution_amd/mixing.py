"""Mixing operators: Python binding of ``include/dwconv_mix.h``.

What a token-mixing block or a separable convolution net has beside its filters
and the operators of ``sequence``:

* ``linear_attention``, ``linear_attention_step``, ``linear_attention_grad``:
  linear attention with a decay for each head;
* ``group_norm``, ``group_norm_grad``: group normalisation with an activation,
  channels last;
* ``quantize_rows``, ``linear_i8``: matrix product in 8-bit integers with a
  scale for each row and each column.

As in ``sequence``: these allocate their outputs and workspace, the
``dwconv_*`` functions mirror the C ABI and write into tensors that the caller
gives; the header states the formulas; calls are asynchronous on ``stream``
(default: the current one of the tensors' device).
"""
import ctypes

from . import sequence as _seq
from .sequence import (_act, _dense, _fits, _gpu, _needed, _rows, _size, _space, _start, _status,
                       _workspace)

T_I8 = 3                     # DWCONV_T_I8
I8_MAX_K = 131071            # DWCONV_I8_MAX_K

ATTENTION_MAX_DIM = 256      # DWCONV_ATTENTION_MAX_DIM

MIX_EXPORTS = ("dwconv_attention_workspace_size", "dwconv_attention_fwd", "dwconv_attention_step",
               "dwconv_attention_grad",
               "dwconv_norm_workspace_size", "dwconv_norm_fwd", "dwconv_norm_grad",
               "dwconv_quantize_rows", "dwconv_linear_i8_workspace_size",
               "dwconv_linear_i8_describe", "dwconv_linear_i8")

__all__ = ["linear_attention", "linear_attention_step", "linear_attention_grad",
           "ATTENTION_MAX_DIM", "group_norm", "group_norm_grad", "quantize_rows", "linear_i8",
           "T_I8", "I8_MAX_K", "MIX_EXPORTS", *MIX_EXPORTS]


def declare(L):
    """Argument types of the entry points of ctypes library L."""
    i, vp, ll, f = ctypes.c_int, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_float
    out = ctypes.POINTER(ll)
    row = [vp, ll]
    seq, heads = [i, ll, vp], [i, i, i, i]
    L.dwconv_attention_workspace_size.argtypes = [i, i, i, ll, i, *heads, out]
    L.dwconv_attention_fwd.argtypes = [*row * 3, i, vp, f, vp, *row, vp, vp, ll, *seq, *heads, vp]
    L.dwconv_attention_step.argtypes = [*row * 3, i, vp, f, vp, *row, i, *heads, vp]
    L.dwconv_attention_grad.argtypes = [*row * 4, i, vp, f, vp, vp, *row * 3, vp, vp, ll, *seq,
                                        *heads, vp]
    L.dwconv_norm_workspace_size.argtypes = [i, i, ll, ll, i, i, out]
    L.dwconv_norm_fwd.argtypes = [*row, i, vp, vp, f, i, *row, vp, vp, ll, ll, ll, i, i, vp]
    L.dwconv_norm_grad.argtypes = [*row * 2, i, vp, vp, i, vp, *row, vp, vp, vp, ll, ll, ll, i, i,
                                   vp]
    L.dwconv_quantize_rows.argtypes = [*row, i, *row, vp, ll, i, vp]
    L.dwconv_linear_i8_workspace_size.argtypes = [i, i, ll, i, i, out]
    L.dwconv_linear_i8_describe.argtypes = [i, i, i, ll, i, i, ctypes.c_char_p, i,
                                            ctypes.POINTER(i)]
    L.dwconv_linear_i8.argtypes = [*row, i, vp, *row, vp, i, vp, i, *row, *row, vp, ll, ll, i, i,
                                   vp]
    for name in MIX_EXPORTS:
        getattr(L, name).restype = i


def _library():
    return _seq._library()


def _code(dtype):
    if _seq.torch is None:
        _seq._setup()
    return T_I8 if dtype is _seq.torch.int8 else _seq._types.get(dtype, -1)


def _is(t, dtype, name):
    if not isinstance(t, _seq.torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")


# ---------------------------- linear attention with a decay for each head
def _flat(t, name, x, shape=None):
    """(address, row stride) of a tensor (..., heads, width) of x's type whose
    rows are its last two axes."""
    if not isinstance(t, _seq.torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t is not x:
        _gpu(t, name, x)
        if t.dtype is not x.dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {x.dtype}")
    if not t.is_contiguous():
        heads, width = t.shape[-2:]
        if (width > 1 and t.stride(-1) != 1) or (heads > 1 and t.stride(-2) != width):
            raise ValueError(f"{name}: the last two axes must be contiguous")
        # a head axis of one may have any stride, which a view of the rows must not see
        t = t.as_strided((*t.shape[:-2], heads * width), (*t.stride()[:-2], 1))
    else:
        return t.data_ptr(), t.shape[-2] * t.shape[-1]
    return _rows(t, name, t)


def _heads(q, k, v, lead):
    """(H, KV, Dk, Dv) of q (..., H, Dk), k (..., KV, Dk) and v (..., KV, Dv), which
    have `lead` leading axes."""
    T = _seq.torch.Tensor
    if not isinstance(k, T) or not isinstance(v, T):
        raise TypeError("k and v must be torch.Tensors")
    if q.dim() != lead + 2:
        raise ValueError(f"q must have {lead + 2} axes here, (..., heads, width)")
    H, Dk = q.shape[-2:]
    if k.dim() != q.dim() or k.shape[:-2] != q.shape[:-2] or k.shape[-1] != Dk:
        raise ValueError("k must be (..., KV heads, Dk) with q's tokens and width")
    KV = k.shape[-2]
    if v.dim() != q.dim() or v.shape[:-1] != k.shape[:-1]:
        raise ValueError("v must be (..., KV heads, Dv) with k's tokens and heads")
    if KV < 1 or H % KV:
        raise ValueError(f"{KV} heads of k and v do not divide the {H} heads of q")
    Dv = v.shape[-1]
    if Dv > _seq._INT_MAX:
        _fits(v, "v")
    return H, KV, Dk, Dv


def _sequences(q, offsets):
    """(sequences, tokens, offsets' address, leading axes) of a dense or packed q."""
    if offsets is None:
        if q.dim() != 4:
            raise ValueError("q must be (sequences, tokens, heads, width), or (tokens, heads, "
                             "width) with offsets")
        return q.shape[0], q.shape[1], None, 2
    if q.dim() != 3:
        raise ValueError("q must be (tokens, heads, width) when offsets are given")
    seqs, tokens, off = _seq._batch(q.select(1, 0), offsets)
    return seqs, tokens, off, 1


def _scale(scale, Dk):
    return Dk ** -0.5 if scale is None else scale


def dwconv_attention_workspace_size(grad, dtype, seqs, tokens, packed, H, KV, Dk, Dv):
    """Workspace bytes of dwconv_attention_fwd (grad false) or dwconv_attention_grad
    (tokens: per sequence, or in all when packed)."""
    return _size("dwconv_attention_workspace_size", int(bool(grad)), _code(dtype), seqs, tokens,
                 int(bool(packed)), H, KV, Dk, Dv)


def dwconv_attention_fwd(q, k, v, log_decay, y, hT=None, workspace=None, scale=None, h0=None,
                         offsets=None, stream=None):
    """y (..., H, Dv) of linear attention; hT receives the last states."""
    code, st, ctx = _start(q, stream, "q")
    if ctx is not None:
        with ctx:
            return dwconv_attention_fwd(q, k, v, log_decay, y, hT, workspace, scale, h0, offsets,
                                        st)
    seqs, tokens, off, lead = _sequences(q, offsets)
    H, KV, Dk, Dv = _heads(q, k, v, lead)
    f32, state = _seq._f32, (seqs, H, Dk, Dv)
    _status(_library().dwconv_attention_fwd(
        *_flat(q, "q", q), *_flat(k, "k", q), *_flat(v, "v", q), code,
        _dense(_needed(log_decay, "log_decay"), "log_decay", q, f32, (H,)), _scale(scale, Dk),
        _dense(h0, "h0", q, f32, state), *_flat(y, "y", q, (*q.shape[:-1], Dv)),
        _dense(hT, "hT", q, f32, state), *_space(workspace, q), seqs, tokens, off, H, KV, Dk, Dv,
        st), "dwconv_attention_fwd")
    return y


def linear_attention(q, k, v, log_decay, h0=None, offsets=None, scale=None, stream=None):
    """(y, hT): linear attention with a decay for each head,

        S = exp(log_decay) * S + k v^T,    y = scale * q S

    token by token within each sequence.  q is (sequences, tokens, H, Dk), or
    (tokens, H, Dk) with offsets, k (..., KV, Dk) and v (..., KV, Dv) alike; KV
    divides H, adjacent query heads sharing a key and value head.  log_decay is
    (H,) float32, at most 0, a constant.  y is (..., H, Dv) of q's type; h0 and
    hT, the states before the first and after the last token, are (sequences, H,
    Dk, Dv) float32.  scale is Dk ** -0.5 by default."""
    _, st, ctx = _start(q, stream, "q")
    if ctx is not None:
        with ctx:
            return linear_attention(q, k, v, log_decay, h0, offsets, scale, st)
    seqs, tokens, off, lead = _sequences(q, offsets)
    H, KV, Dk, Dv = _heads(q, k, v, lead)
    ws = _workspace(dwconv_attention_workspace_size(False, q.dtype, seqs, tokens, off is not None,
                                                    H, KV, Dk, Dv), q)
    y = q.new_empty((*q.shape[:-1], Dv))
    hT = q.new_empty((seqs, H, Dk, Dv), dtype=_seq._f32)
    dwconv_attention_fwd(q, k, v, log_decay, y, hT, ws, scale, h0, offsets, st)
    return y, hT


def dwconv_attention_step(q, k, v, log_decay, h, y, scale=None, stream=None):
    """One token for each sequence; h (sequences, H, Dk, Dv) float32 in place."""
    code, st, ctx = _start(q, stream, "q")
    if ctx is not None:
        with ctx:
            return dwconv_attention_step(q, k, v, log_decay, h, y, scale, st)
    H, KV, Dk, Dv = _heads(q, k, v, 1)
    seqs, f32 = q.shape[0], _seq._f32
    _status(_library().dwconv_attention_step(
        *_flat(q, "q", q), *_flat(k, "k", q), *_flat(v, "v", q), code,
        _dense(_needed(log_decay, "log_decay"), "log_decay", q, f32, (H,)), _scale(scale, Dk),
        _dense(_needed(h, "h"), "h", q, f32, (seqs, H, Dk, Dv)),
        *_flat(y, "y", q, (seqs, H, Dv)), seqs, H, KV, Dk, Dv, st), "dwconv_attention_step")
    return y


def linear_attention_step(q, k, v, log_decay, h, scale=None, stream=None):
    """y (sequences, H, Dv) for one token of each sequence, q (sequences, H, Dk);
    the states h (sequences, H, Dk, Dv) float32 are updated in place."""
    _, st, ctx = _start(q, stream, "q")
    if ctx is not None:
        with ctx:
            return linear_attention_step(q, k, v, log_decay, h, scale, st)
    _, _, _, Dv = _heads(q, k, v, 1)
    return dwconv_attention_step(q, k, v, log_decay, h, q.new_empty((*q.shape[:-1], Dv)), scale,
                                 st)


def dwconv_attention_grad(dy, q, k, v, log_decay, dq, dk, dv, dh0=None, workspace=None, scale=None,
                          h0=None, dhT=None, offsets=None, stream=None):
    """Gradients of linear_attention into dq, dk, dv and dh0, each of which may be None."""
    code, st, ctx = _start(q, stream, "q")
    if ctx is not None:
        with ctx:
            return dwconv_attention_grad(dy, q, k, v, log_decay, dq, dk, dv, dh0, workspace,
                                         scale, h0, dhT, offsets, st)
    seqs, tokens, off, lead = _sequences(q, offsets)
    H, KV, Dk, Dv = _heads(q, k, v, lead)
    f32, state = _seq._f32, (seqs, H, Dk, Dv)
    out = [(None, 0) if t is None else _flat(t, name, q, like.shape)
           for t, name, like in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v))]
    _status(_library().dwconv_attention_grad(
        *_flat(dy, "dy", q, (*q.shape[:-1], Dv)), *_flat(q, "q", q), *_flat(k, "k", q),
        *_flat(v, "v", q), code, _dense(_needed(log_decay, "log_decay"), "log_decay", q, f32,
                                        (H,)), _scale(scale, Dk),
        _dense(h0, "h0", q, f32, state), _dense(dhT, "dhT", q, f32, state), *out[0], *out[1],
        *out[2], _dense(dh0, "dh0", q, f32, state), *_space(workspace, q), seqs, tokens, off, H,
        KV, Dk, Dv, st), "dwconv_attention_grad")
    return dq, dk, dv, dh0


def linear_attention_grad(dy, q, k, v, log_decay, h0=None, dhT=None, offsets=None, scale=None,
                          stream=None):
    """(dq, dk, dv, dh0) of linear_attention for the cotangents dy of y and dhT (or
    None) of hT.  dh0 (sequences, H, Dk, Dv) float32 is None unless h0 is given."""
    _, st, ctx = _start(q, stream, "q")
    if ctx is not None:
        with ctx:
            return linear_attention_grad(dy, q, k, v, log_decay, h0, dhT, offsets, scale, st)
    seqs, tokens, off, lead = _sequences(q, offsets)
    H, KV, Dk, Dv = _heads(q, k, v, lead)
    ws = _workspace(dwconv_attention_workspace_size(True, q.dtype, seqs, tokens, off is not None,
                                                    H, KV, Dk, Dv), q)
    dq, dk, dv = (q.new_empty(t.shape) for t in (q, k, v))
    dh0 = None if h0 is None else q.new_empty((seqs, H, Dk, Dv), dtype=_seq._f32)
    return dwconv_attention_grad(dy, q, k, v, log_decay, dq, dk, dv, dh0, ws, scale, h0, dhT,
                                 offsets, st)


# ------------------------------- group normalisation with an activation
def _instances(x, groups):
    """(instances, positions, channels) of a channels-last tensor."""
    if x.dim() < 2:
        raise ValueError("x must be (instances, ..., channels)")
    C = x.shape[-1]
    if isinstance(groups, bool) or not isinstance(groups, int):
        raise TypeError("groups must be an int")
    if abs(groups) > _seq._INT_MAX:
        raise ValueError(f"{groups} groups of {C} channels")
    P = 1
    for size in x.shape[1:-1]:
        P *= size
    return x.shape[0], P, C


def dwconv_norm_workspace_size(grad, dtype, N, P, C, groups):
    """Workspace bytes of dwconv_norm_fwd (grad false) or dwconv_norm_grad."""
    return _size("dwconv_norm_workspace_size", int(bool(grad)), _code(dtype), N, P, C, groups)


def dwconv_norm_fwd(x, groups, w, b, y, eps=1e-5, act="none", stats=None, workspace=None,
                    stream=None):
    """y = act(x normalised over each group * w + b); stats receives (mean, rstd)."""
    code, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return dwconv_norm_fwd(x, groups, w, b, y, eps, act, stats, workspace, st)
    N, P, C = _instances(x, groups)
    f32 = _seq._f32
    _status(_library().dwconv_norm_fwd(
        *_rows(x, "x", x), code, _dense(w, "w", x, f32, (C,)), _dense(b, "b", x, f32, (C,)), eps,
        _act(act), *_rows(y, "y", x, x.shape), _dense(stats, "stats", x, f32, (N, groups, 2)),
        *_space(workspace, x), N, P, C, groups, st), "dwconv_norm_fwd")
    return y


def group_norm(x, groups, w=None, b=None, eps=1e-5, act="none", save_stats=False, stream=None):
    """y = act((x - mean) * rstd * w + b), or (y, stats) with save_stats: x (N, ...,
    C) normalised over the positions (one at least) and the C / groups adjacent channels of
    each group of each of the N instances.  A tensor of tokens, (tokens, C), is
    normalised token by token.  w and b are (C,) float32; stats (N, groups, 2)
    float32, mean and rstd, is what group_norm_grad needs."""
    _, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return group_norm(x, groups, w, b, eps, act, save_stats, st)
    N, P, C = _instances(x, groups)
    ws = _workspace(dwconv_norm_workspace_size(False, x.dtype, N, P, C, groups), x)
    y = x.new_empty(x.shape)
    stats = x.new_empty((N, groups, 2), dtype=_seq._f32) if save_stats else None
    dwconv_norm_fwd(x, groups, w, b, y, eps, act, stats, ws, st)
    return (y, stats) if save_stats else y


def dwconv_norm_grad(dy, x, stats, groups, w, b, dx, dw, db, act="none", workspace=None,
                     stream=None):
    """Gradients of group_norm into dx, dw and db, each of which may be None."""
    code, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return dwconv_norm_grad(dy, x, stats, groups, w, b, dx, dw, db, act, workspace, st)
    N, P, C = _instances(x, groups)
    f32 = _seq._f32
    _status(_library().dwconv_norm_grad(
        *_rows(dy, "dy", x, x.shape), *_rows(x, "x", x), code, _dense(w, "w", x, f32, (C,)),
        _dense(b, "b", x, f32, (C,)), _act(act),
        _dense(_needed(stats, "stats"), "stats", x, f32, (N, groups, 2)),
        *((None, 0) if dx is None else _rows(dx, "dx", x, x.shape)),
        _dense(dw, "dw", x, f32, (C,)), _dense(db, "db", x, f32, (C,)), *_space(workspace, x), N,
        P, C, groups, st), "dwconv_norm_grad")
    return dx, dw, db


def group_norm_grad(dy, x, stats, groups, w=None, b=None, act="none", stream=None):
    """(dx, dw, db) of group_norm for the cotangent dy of y; stats are those that
    group_norm kept.  dw and db are (C,) float32."""
    _, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return group_norm_grad(dy, x, stats, groups, w, b, act, st)
    N, P, C = _instances(x, groups)
    ws = _workspace(dwconv_norm_workspace_size(True, x.dtype, N, P, C, groups), x)
    dx = x.new_empty(x.shape)
    dw, db = x.new_empty((C,), dtype=_seq._f32), x.new_empty((C,), dtype=_seq._f32)
    return dwconv_norm_grad(dy, x, stats, groups, w, b, dx, dw, db, act, ws, st)


# ------------------------------------------ matrix product in 8-bit integers
def dwconv_quantize_rows(x, q, scale, stream=None):
    """q (..., K) int8 and scale (...) float32 of the rows of x (..., K)."""
    code, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return dwconv_quantize_rows(x, q, scale, st)
    K = x.shape[-1]
    _is(q, _seq.torch.int8, "q")
    _gpu(q, "q", x)
    if q.shape != x.shape:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected {tuple(x.shape)}")
    _status(_library().dwconv_quantize_rows(
        *_rows(x, "x", x), code, *_rows(q, "q", q),
        _dense(_needed(scale, "scale"), "scale", x, _seq._f32, x.shape[:-1]),
        x.numel() // max(K, 1), K, st), "dwconv_quantize_rows")
    return q, scale


def quantize_rows(x, stream=None):
    """(q, scale): the rows of x (..., K) as int8 numbers (..., K) and float32
    scales (...), scale = max |x| * (1 / 127), factor and product rounded to float32 (up to
    one unit in the last place from max |x| / 127), and q = x / scale, rounded to the nearest
    integer.  A row that is not finite has the scale NaN and numbers of 0."""
    _, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return quantize_rows(x, st)
    if x.dim() < 1:
        raise ValueError("x must have at least one axis")
    q = x.new_empty(x.shape, dtype=_seq.torch.int8)
    scale = x.new_empty(x.shape[:-1], dtype=_seq._f32)
    return dwconv_quantize_rows(x, q, scale, st)


def dwconv_linear_i8_workspace_size(xdtype, dtype, M, N, K):
    """Workspace bytes of dwconv_linear_i8 for x of xdtype (int8, or dtype)."""
    return _size("dwconv_linear_i8_workspace_size", _code(xdtype), _code(dtype), M, N, K)


def dwconv_linear_i8_describe(quantized, dtype, M, N, K, aligned=True):
    """(kernel, ranges of the summed index) of the product."""
    name, splits = ctypes.create_string_buffer(64), ctypes.c_int(0)
    _status(_library().dwconv_linear_i8_describe(
        int(bool(quantized)), _code(dtype), int(bool(aligned)), M, N, K, name, 64,
        ctypes.byref(splits)), "dwconv_linear_i8_describe")
    return name.value.decode(), splits.value


def dwconv_linear_i8(x, w, w_scale, b, y, act="none", res=None, x_scale=None, workspace=None,
                     stream=None):
    """y = act(x_scale w_scale x w^T + b) + res; x int8, or y's type and quantised here."""
    code, st, ctx = _start(y, stream, "y")
    if ctx is not None:
        with ctx:
            return dwconv_linear_i8(x, w, w_scale, b, y, act, res, x_scale, workspace, st)
    t = _seq.torch
    N, K = _map(x, w)
    _gpu(x, "x", y)
    _gpu(w, "w", y)
    if x.dtype is not (t.int8 if x_scale is not None else y.dtype):
        raise TypeError(f"x has dtype {x.dtype}, expected {y.dtype}, or int8 with x_scale")
    shape = (*x.shape[:-1], N)
    if y.shape != shape:
        raise ValueError(f"y has shape {tuple(y.shape)}, expected {shape}")
    _status(_library().dwconv_linear_i8(
        *_rows(x, "x", x), T_I8 if x_scale is not None else code,
        _dense(x_scale, "x_scale", y, _seq._f32, x.shape[:-1]), *_rows(w, "w", w),
        _dense(_needed(w_scale, "w_scale"), "w_scale", y, _seq._f32, (N,)), code,
        _dense(b, "b", y, _seq._f32, (N,)), _act(act),
        *((None, 0) if res is None else _rows(res, "res", y, shape)),
        *_rows(y, "y", y), *_space(workspace, y),
        x.numel() // max(K, 1), N, K, st), "dwconv_linear_i8")
    return y


def _map(x, w):
    """(N, K) of a linear map w of x."""
    t = _seq.torch
    _is(w, t.int8, "w")
    if not isinstance(x, t.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dim() < 1 or w.dim() != 2 or w.shape[1] != x.shape[-1]:
        raise ValueError("w must be (N, K) with K the last axis of x")
    N, K = w.shape
    if N > _seq._INT_MAX:
        _fits(w, "w")
    return N, K


def linear_i8(x, w, w_scale, b=None, act="none", res=None, x_scale=None, dtype=None, stream=None):
    """y = act(x_scale w_scale x w^T + b) + res in 8-bit integers: ``linear`` for
    serving.  w (N, K) int8 and w_scale (N,) float32 are a matrix's
    quantize_rows; b is (N,) float32.  x (..., K) is float32, float16 or bfloat16
    and quantised here, row by row, with y and res of its type; or it is int8
    with its x_scale, with y of `dtype` (default: res's type)."""
    if _seq.torch is None:
        _seq._setup()
    if x_scale is None:
        anchor = x
        if dtype is not None and isinstance(x, _seq.torch.Tensor) and x.dtype is not dtype:
            raise TypeError(f"x has dtype {x.dtype}, expected {dtype}, or int8 with x_scale")
    else:
        anchor = x_scale
        if dtype is None:
            if res is None:
                raise TypeError("dtype is needed for an int8 x without res")
            dtype = res.dtype
        if _code(dtype) not in (0, 1, 2):
            raise TypeError(f"dtype is {dtype}, expected float32, float16 or bfloat16")
    _, st, ctx = _start(anchor, stream, "x" if x_scale is None else "x_scale")
    if ctx is not None:
        with ctx:
            return linear_i8(x, w, w_scale, b, act, res, x_scale, dtype, st)
    N, K = _map(x, w)
    y = anchor.new_empty((*x.shape[:-1], N), dtype=dtype or x.dtype)
    ws = _workspace(dwconv_linear_i8_workspace_size(x.dtype, y.dtype, x.numel() // max(K, 1), N,
                                                    K), y)
    return dwconv_linear_i8(x, w, w_scale, b, y, act, res, x_scale, ws, st)
