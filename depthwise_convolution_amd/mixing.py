"""Mixing operators: Python binding of ``include/dwconv_mix.h``.

What a token-mixing block or a separable convolution net has beside its filters
and the operators of ``sequence``:

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
from .sequence import (_act, _dense, _gpu, _needed, _rows, _size, _space, _start, _status,
                       _workspace)

T_I8 = 3                     # DWCONV_T_I8
I8_MAX_K = 131071            # DWCONV_I8_MAX_K

MIX_EXPORTS = ("dwconv_norm_workspace_size", "dwconv_norm_fwd", "dwconv_norm_grad",
               "dwconv_quantize_rows", "dwconv_linear_i8_workspace_size",
               "dwconv_linear_i8_describe", "dwconv_linear_i8")

__all__ = ["group_norm", "group_norm_grad", "quantize_rows", "linear_i8", "T_I8", "I8_MAX_K", "MIX_EXPORTS", *MIX_EXPORTS]


def declare(L):
    """Argument types of the entry points of ctypes library L."""
    i, vp, ll, f = ctypes.c_int, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_float
    out = ctypes.POINTER(ll)
    row = [vp, ll]
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


# ------------------------------- group normalisation with an activation
def _instances(x, groups):
    """(instances, positions, channels) of a channels-last tensor."""
    if x.dim() < 2:
        raise ValueError("x must be (instances, ..., channels)")
    C = x.shape[-1]
    if isinstance(groups, bool) or not isinstance(groups, int):
        raise TypeError("groups must be an int")
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
    C) normalised over the positions and the C / groups adjacent channels of each
    group of each of the N instances.  A tensor of tokens, (tokens, C), is
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
    scales (...), scale = max |x| / 127 and q = x / scale, rounded to the nearest
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
    return w.shape


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
