"""Sequence operators: Python binding of ``include/dwconv_seq.h``.

The parts of a recurrent token-mixing block around the depthwise filter:

* ``causal_conv``, ``causal_conv_step``, ``causal_conv_grad``: causal
  depthwise convolution over tokens with carried rows;
* ``gated_scan``, ``gated_scan_step``, ``gated_scan_grad``: gated linear
  recurrence;
* ``linear``, ``linear_grad``: matrix product with bias, activation and
  residual.

These allocate their outputs and workspace; the ``dwconv_*`` functions mirror
the C ABI and write into tensors that the caller gives.  The header states the
formulas.

Activations are float32, float16 or bfloat16 (``x.dtype``).  A batch is dense,
``(sequences, tokens, C)``, or packed, ``(tokens, C)`` with ``offsets``, an
int32 GPU tensor of ``sequences + 1`` row numbers from 0 to ``tokens``; the
single-token forms take ``(sequences, C)``.  The last axis is contiguous; rows
may be strided (a column range of a wider tensor) as long as they are evenly
spaced.

Calls are asynchronous on ``stream`` (default: the current one of the tensors'
device); outputs and workspaces made here are allocated on that stream.
Tensors that another stream works on are the caller's to order, as with any
PyTorch operator.
"""
import ctypes

torch = None                 # imported by the first call

T_F32, T_F16, T_BF16 = 0, 1, 2
CAUSAL_MAX_TAPS = 8          # DWCONV_CAUSAL_MAX_TAPS
SEQ_MAX_ROWS = (1 << 31) - (1 << 16)         # DWCONV_SEQ_MAX_ROWS
SCAN_RUN = 8                # DWCONV_SCAN_RUN
LINEAR_Y, LINEAR_DX, LINEAR_DW = 0, 1, 2     # DWCONV_LINEAR_*

SEQ_EXPORTS = ("dwconv_causal_fwd", "dwconv_causal_step", "dwconv_causal_grad_workspace_size",
               "dwconv_causal_grad", "dwconv_scan_states_size", "dwconv_scan_workspace_size",
               "dwconv_scan_fwd", "dwconv_scan_step", "dwconv_scan_grad",
               "dwconv_linear_workspace_size", "dwconv_linear_describe", "dwconv_linear_fwd",
               "dwconv_linear_grad")

__all__ = ["causal_conv", "causal_conv_step", "causal_conv_grad", "gated_scan",
           "gated_scan_step", "gated_scan_grad", "linear", "linear_grad", "T_F32", "T_F16",
           "T_BF16", "CAUSAL_MAX_TAPS", "SEQ_MAX_ROWS", "SCAN_RUN", "LINEAR_Y", "LINEAR_DX",
           "LINEAR_DW", "SEQ_EXPORTS", *SEQ_EXPORTS]


def declare(L):
    """Argument types of the entry points of ctypes library L."""
    i, vp, ll, f = ctypes.c_int, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_float
    out = ctypes.POINTER(ll)
    row = [vp, ll]
    seq = [i, ll, vp]
    L.dwconv_causal_fwd.argtypes = [*row, i, vp, i, vp, i, vp, *row, vp, *seq, i, i, vp]
    L.dwconv_causal_step.argtypes = [*row, i, vp, i, vp, i, vp, *row, i, i, i, vp]
    L.dwconv_causal_grad_workspace_size.argtypes = [i, ll, i, i, i, out]
    L.dwconv_causal_grad.argtypes = [*row, *row, i, vp, i, vp, i, vp, vp, *row, vp, vp, vp,
                                     vp, ll, *seq, i, i, vp]
    L.dwconv_scan_states_size.argtypes = [i, ll, i, i, out]
    L.dwconv_scan_workspace_size.argtypes = [i, i, ll, i, i, out]
    L.dwconv_scan_fwd.argtypes = [*row * 3, i, vp, f, vp, *row, vp, vp, vp, ll, *seq, i, vp]
    L.dwconv_scan_step.argtypes = [*row * 3, i, vp, f, vp, *row, i, i, vp]
    L.dwconv_scan_grad.argtypes = [*row * 4, i, vp, f, vp, vp, *row * 3, vp, vp, vp, ll, *seq, i,
                                   vp]
    L.dwconv_linear_workspace_size.argtypes = [i, i, i, ll, i, i, out]
    L.dwconv_linear_describe.argtypes = [i, i, i, ll, i, i, ctypes.c_char_p, i,
                                         ctypes.POINTER(i)]
    L.dwconv_linear_fwd.argtypes = [*row * 2, i, vp, i, *row * 3, vp, ll, ll, i, i, vp]
    L.dwconv_linear_grad.argtypes = [*row * 3, i, i, *row * 3, vp, vp, ll, ll, i, i, vp]
    for name in SEQ_EXPORTS:
        getattr(L, name).restype = i


# ---------------------------------------------------------------- marshalling
# A call for a single token takes a few microseconds on the GPU, so what happens
# before it is kept short: one pass of checks, no object per argument.
_pkg = _types = _acts = _f32 = _raw_stream = None
_many_devices = False


class _Handle(int):
    """A hipStream_t whose device and stream are the current ones."""


def _setup():
    global torch, _pkg, _types, _acts, _f32, _raw_stream, _many_devices
    import torch as t

    import depthwise_convolution_amd as pkg
    _types = {t.float32: T_F32, t.float16: T_F16, t.bfloat16: T_BF16}
    _acts = {"none": pkg.ACT_NONE, "relu": pkg.ACT_RELU, "relu6": pkg.ACT_RELU6,
             "silu": pkg.ACT_SILU}
    _f32 = t.float32
    _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream",
                          lambda index: t.cuda.current_stream(index).cuda_stream)
    _many_devices = t.cuda.is_available() and t.cuda.device_count() > 1
    _pkg, torch = pkg, t


def _library():
    if torch is None:
        _setup()
    return _pkg._lib or _pkg.lib()


def _act(act):
    code = _acts.get(act) if isinstance(act, str) else None
    return _pkg._act_code(act) if code is None else code


def _start(x, stream, name="x"):
    """(x's type code, stream handle, context or None) of a call.  Where there is
    a context, the call is made again inside it, with the handle as its stream:
    then the tensors' device and stream are the current ones, and what is
    allocated belongs to the stream."""
    if torch is None:
        _setup()
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not x.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")
    code = _types.get(x.dtype)
    if code is None:
        raise TypeError(f"{name} has dtype {x.dtype}, expected float32, float16 or bfloat16")
    if type(stream) is _Handle:
        return code, stream, None
    index = x.get_device()
    if stream is None:
        handle = _Handle(_raw_stream(index))
        away = _many_devices and index != torch.cuda.current_device()
        return code, handle, torch.cuda.device(index) if away else None
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=x.device)
    elif getattr(stream, "device", x.device) != x.device:
        raise ValueError(f"stream is on {stream.device}, {name} on {x.device}")
    return code, _Handle(stream.cuda_stream), torch.cuda.stream(stream)


def _gpu(t, name, x):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != x.get_device():
        raise ValueError(f"{name} must be on the GPU device of x")


def _rows(t, name, x, shape=None):
    """(address, row stride) of a tensor of x's type whose rows are its last axis."""
    if t is not x:
        _gpu(t, name, x)
        if t.dtype is not x.dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {x.dtype}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return t.data_ptr(), t.shape[-1]
    width = t.shape[-1]
    if width > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    # leading axes longer than one, from the innermost: evenly spaced rows
    ld = count = None
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if ld is None:
            ld, count = stride, size
        elif stride == ld * count:
            count *= size
        else:
            raise ValueError(f"{name}: rows must be evenly spaced")
    if ld is None:
        ld = width
    if ld < width:
        raise ValueError(f"{name}: rows overlap")
    return t.data_ptr(), ld


def _dense(t, name, x, dtype, shape):
    """Address of a dense tensor (None: NULL)."""
    if t is None:
        return None
    _gpu(t, name, x)
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _needed(t, name):
    if t is None:
        raise TypeError(f"{name} must be a torch.Tensor")
    return t


def _batch(x, offsets):
    """(sequences, tokens, offsets' address) of a dense or packed batch."""
    if offsets is None:
        if x.dim() != 3:
            raise ValueError("x must be (sequences, tokens, C), or (tokens, C) with offsets")
        return x.shape[0], x.shape[1], None
    if x.dim() != 2:
        raise ValueError("x must be (tokens, C) when offsets are given")
    _gpu(offsets, "offsets", x)
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.numel() < 2 \
            or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous int32 tensor of sequences + 1 numbers")
    return offsets.numel() - 1, x.shape[0], offsets.data_ptr()


def _tokens(x):
    if x.dim() != 2:
        raise ValueError("x must be (sequences, C)")
    return x.shape


def _filter(w, x):
    """(address, type code, taps) of a filter."""
    _gpu(w, "w", x)
    code = _types.get(w.dtype)
    if code is None:
        raise TypeError(f"w has dtype {w.dtype}, expected float32, float16 or bfloat16")
    if w.dim() != 2 or w.shape[0] != x.shape[-1] or not w.is_contiguous():
        raise ValueError("w must be a contiguous (C, taps) tensor")
    return w.data_ptr(), code, w.shape[1]


def _weights(w, x):
    """(address, row stride, N, K) of a linear map."""
    pw, ldw = _rows(w, "w", x)
    if w.dim() != 2 or w.shape[1] != x.shape[-1]:
        raise ValueError("w must be (N, K) with K the last axis of x")
    return pw, ldw, w.shape[0], w.shape[1]


def _status(st, what):
    if st != 0:
        raise _pkg.DwconvError(st, what)


def _size(what, *args):
    out = ctypes.c_longlong(0)
    _status(getattr(_library(), what)(*args, ctypes.byref(out)), what)
    return out.value


def _workspace(nbytes, x):
    return x.new_empty(nbytes, dtype=torch.uint8) if nbytes else None


def _space(ws, x):
    """(address, bytes) of a workspace (None: NULL)."""
    if ws is None:
        return None, 0
    _gpu(ws, "workspace", x)
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


# ------------------------------------------- causal depthwise convolution
def dwconv_causal_fwd(x, w, b, y, act="none", init=None, final=None, offsets=None, stream=None):
    """y = act(causal filter w of x, plus b); final receives the rows to carry."""
    code, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return dwconv_causal_fwd(x, w, b, y, act, init, final, offsets, st)
    seqs, tokens, off = _batch(x, offsets)
    C = x.shape[-1]
    px, ldx = _rows(x, "x", x)
    pw, wt, K = _filter(w, x)
    py, ldy = _rows(y, "y", x, x.shape)
    carried = (seqs, K - 1, C)
    _status(_library().dwconv_causal_fwd(
        px, ldx, code, pw, wt, _dense(b, "b", x, _f32, (C,)), _act(act),
        _dense(init, "init", x, x.dtype, carried), py, ldy,
        _dense(final, "final", x, x.dtype, carried), seqs, tokens, off, C, K, st),
        "dwconv_causal_fwd")
    return y


def causal_conv(x, w, b=None, act="none", init=None, offsets=None, stream=None):
    """(y, final): y = act(b + causal filter w of x), and the taps - 1 rows of
    each sequence that a continuation passes as init.

    w is (C, taps) of any of the types, b (C,) float32, init and final
    (sequences, taps - 1, C) of x's type, the oldest row first."""
    _, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return causal_conv(x, w, b, act, init, offsets, st)
    seqs, _, _ = _batch(x, offsets)
    _, _, K = _filter(w, x)
    y = x.new_empty(x.shape)
    final = x.new_empty((seqs, K - 1, x.shape[-1]))
    dwconv_causal_fwd(x, w, b, y, act, init, final, offsets, st)
    return y, final


def dwconv_causal_step(x, w, b, state, y, act="none", stream=None):
    """One token for each sequence; state (sequences, taps - 1, C) in place."""
    code, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return dwconv_causal_step(x, w, b, state, y, act, st)
    seqs, C = _tokens(x)
    px, ldx = _rows(x, "x", x)
    pw, wt, K = _filter(w, x)
    py, ldy = _rows(y, "y", x, x.shape)
    _status(_library().dwconv_causal_step(
        px, ldx, code, pw, wt, _dense(b, "b", x, _f32, (C,)), _act(act),
        _dense(state, "state", x, x.dtype, (seqs, K - 1, C)), py, ldy, seqs, C, K, st),
        "dwconv_causal_step")
    return y


def causal_conv_step(x, state, w, b=None, act="none", stream=None):
    """y (sequences, C) for one token of each sequence; state is updated in place."""
    _, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return causal_conv_step(x, state, w, b, act, st)
    return dwconv_causal_step(x, w, b, state, x.new_empty(x.shape), act, st)


def dwconv_causal_grad_workspace_size(seqs, tokens, packed, C, K):
    """Workspace bytes of dwconv_causal_grad (tokens: per sequence, or in all when packed)."""
    return _size("dwconv_causal_grad_workspace_size", seqs, tokens, int(bool(packed)), C, K)


def dwconv_causal_grad(dy, x, w, b, dx, dw, db, workspace, act="none", init=None, dfinal=None,
                       dinit=None, offsets=None, stream=None):
    """Gradients of causal_conv into dx, dw, db (or None) and dinit (or None)."""
    code, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return dwconv_causal_grad(dy, x, w, b, dx, dw, db, workspace, act, init, dfinal,
                                      dinit, offsets, st)
    seqs, tokens, off = _batch(x, offsets)
    C, kind = x.shape[-1], x.dtype
    pw, wt, K = _filter(w, x)
    carried = (seqs, K - 1, C)
    _status(_library().dwconv_causal_grad(
        *_rows(dy, "dy", x, x.shape), *_rows(x, "x", x), code, pw, wt,
        _dense(b, "b", x, _f32, (C,)), _act(act), _dense(init, "init", x, kind, carried),
        _dense(dfinal, "dfinal", x, kind, carried), *_rows(dx, "dx", x, x.shape),
        _dense(_needed(dw, "dw"), "dw", x, _f32, (C, K)), _dense(db, "db", x, _f32, (C,)),
        _dense(dinit, "dinit", x, kind, carried), *_space(workspace, x), seqs, tokens, off, C, K,
        st), "dwconv_causal_grad")
    return dx, dw, db, dinit


def causal_conv_grad(dy, x, w, b=None, act="none", init=None, dfinal=None, offsets=None,
                     stream=None):
    """(dx, dw, db, dinit) of causal_conv for the cotangents dy of y and dfinal
    (or None) of final.  dw (C, taps) and db (C,) are float32; dinit is None
    unless init is given."""
    _, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return causal_conv_grad(dy, x, w, b, act, init, dfinal, offsets, st)
    seqs, tokens, off = _batch(x, offsets)
    _, _, K = _filter(w, x)
    C = x.shape[-1]
    dx = x.new_empty(x.shape)
    dw = x.new_empty((C, K), dtype=_f32)
    db = x.new_empty((C,), dtype=_f32)
    dinit = None if init is None else x.new_empty((seqs, K - 1, C))
    ws = _workspace(dwconv_causal_grad_workspace_size(seqs, tokens, off is not None, C, K), x)
    return dwconv_causal_grad(dy, x, w, b, dx, dw, db, ws, act, init, dfinal, dinit, offsets, st)


# ------------------------------------------------- gated linear recurrence
def dwconv_scan_states_size(seqs, tokens, packed, C):
    """Floats that dwconv_scan_fwd keeps for the gradient."""
    return _size("dwconv_scan_states_size", seqs, tokens, int(bool(packed)), C)


def dwconv_scan_workspace_size(grad, seqs, tokens, packed, C):
    """Workspace bytes of dwconv_scan_fwd (grad false) or dwconv_scan_grad."""
    return _size("dwconv_scan_workspace_size", int(bool(grad)), seqs, tokens, int(bool(packed)),
                 C)


def _states(states, x, seqs, tokens, packed):
    if states is None:
        return None
    C = x.shape[-1]
    return _dense(states, "states", x, _f32, (dwconv_scan_states_size(seqs, tokens, packed, C),))


def dwconv_scan_fwd(x, r, i, lam, y, hT=None, states=None, workspace=None, scale=8.0, h0=None,
                    offsets=None, stream=None):
    """y = the states of the recurrence; hT the last ones; states for the gradient."""
    code, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return dwconv_scan_fwd(x, r, i, lam, y, hT, states, workspace, scale, h0, offsets,
                                   st)
    seqs, tokens, off = _batch(x, offsets)
    C, shape = x.shape[-1], x.shape
    _status(_library().dwconv_scan_fwd(
        *_rows(x, "x", x), *_rows(r, "r", x, shape), *_rows(i, "i", x, shape), code,
        _dense(_needed(lam, "lam"), "lam", x, _f32, (C,)), scale,
        _dense(h0, "h0", x, _f32, (seqs, C)), *_rows(y, "y", x, shape),
        _dense(hT, "hT", x, _f32, (seqs, C)), _states(states, x, seqs, tokens, off is not None),
        *_space(workspace, x), seqs, tokens, off, C, st), "dwconv_scan_fwd")
    return y


def gated_scan(x, r, i, lam, h0=None, offsets=None, scale=8.0, save_states=False, stream=None):
    """(y, hT), or (y, hT, states) with save_states: the gated recurrence

        h = a * h + sqrt(1 - a^2) * sigmoid(i) * x,
        log a = -scale * softplus(lam) * sigmoid(r)

    per channel, y its states in x's type, hT (sequences, C) float32 the last
    ones, states what gated_scan_grad needs.  r and i are the gates before
    their sigmoid, shaped as x; lam is (C,), h0 (sequences, C), both float32."""
    _, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return gated_scan(x, r, i, lam, h0, offsets, scale, save_states, st)
    seqs, tokens, off = _batch(x, offsets)
    C, packed = x.shape[-1], off is not None
    y = x.new_empty(x.shape)
    hT = x.new_empty((seqs, C), dtype=_f32)
    states = None
    if save_states:
        states = x.new_empty((dwconv_scan_states_size(seqs, tokens, packed, C),), dtype=_f32)
    ws = _workspace(dwconv_scan_workspace_size(False, seqs, tokens, packed, C), x)
    dwconv_scan_fwd(x, r, i, lam, y, hT, states, ws, scale, h0, offsets, st)
    return (y, hT, states) if save_states else (y, hT)


def dwconv_scan_step(x, r, i, lam, h, y, scale=8.0, stream=None):
    """One token for each sequence; h (sequences, C) float32 in place."""
    code, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return dwconv_scan_step(x, r, i, lam, h, y, scale, st)
    seqs, C = shape = _tokens(x)
    _status(_library().dwconv_scan_step(
        *_rows(x, "x", x), *_rows(r, "r", x, shape), *_rows(i, "i", x, shape), code,
        _dense(_needed(lam, "lam"), "lam", x, _f32, (C,)), scale,
        _dense(_needed(h, "h"), "h", x, _f32, shape), *_rows(y, "y", x, shape), seqs, C, st),
        "dwconv_scan_step")
    return y


def gated_scan_step(x, r, i, lam, h, scale=8.0, stream=None):
    """y (sequences, C) for one token of each sequence; h is updated in place."""
    _, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return gated_scan_step(x, r, i, lam, h, scale, st)
    return dwconv_scan_step(x, r, i, lam, h, x.new_empty(x.shape), scale, st)


def dwconv_scan_grad(dy, x, r, i, lam, states, dx, dr, di, dlam, dh0=None, workspace=None,
                     scale=8.0, dhT=None, offsets=None, stream=None):
    """Gradients of gated_scan into dx, dr, di, dlam and dh0 (or None)."""
    code, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return dwconv_scan_grad(dy, x, r, i, lam, states, dx, dr, di, dlam, dh0, workspace,
                                    scale, dhT, offsets, st)
    seqs, tokens, off = _batch(x, offsets)
    C, shape = x.shape[-1], x.shape
    _status(_library().dwconv_scan_grad(
        *_rows(dy, "dy", x, shape), *_rows(x, "x", x), *_rows(r, "r", x, shape),
        *_rows(i, "i", x, shape), code, _dense(_needed(lam, "lam"), "lam", x, _f32, (C,)), scale,
        _states(_needed(states, "states"), x, seqs, tokens, off is not None),
        _dense(dhT, "dhT", x, _f32, (seqs, C)), *_rows(dx, "dx", x, shape),
        *_rows(dr, "dr", x, shape), *_rows(di, "di", x, shape),
        _dense(_needed(dlam, "dlam"), "dlam", x, _f32, (C,)),
        _dense(dh0, "dh0", x, _f32, (seqs, C)), *_space(workspace, x), seqs, tokens, off, C, st),
        "dwconv_scan_grad")
    return dx, dr, di, dlam, dh0


def gated_scan_grad(dy, x, r, i, lam, states, dhT=None, offsets=None, scale=8.0, stream=None):
    """(dx, dr, di, dlam, dh0) of gated_scan for the cotangents dy of y and dhT
    (or None) of hT; states are those that gated_scan kept.  dlam (C,) and dh0
    (sequences, C) are float32."""
    _, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return gated_scan_grad(dy, x, r, i, lam, states, dhT, offsets, scale, st)
    seqs, tokens, off = _batch(x, offsets)
    C = x.shape[-1]
    dx, dr, di = (x.new_empty(x.shape) for _ in range(3))
    dlam = x.new_empty((C,), dtype=_f32)
    dh0 = x.new_empty((seqs, C), dtype=_f32)
    ws = _workspace(dwconv_scan_workspace_size(True, seqs, tokens, off is not None, C), x)
    return dwconv_scan_grad(dy, x, r, i, lam, states, dx, dr, di, dlam, dh0, ws, scale, dhT,
                            offsets, st)


# --------------------------------- matrix product with bias, activation, residual
def dwconv_linear_workspace_size(grad, dtype, act, M, N, K):
    """Workspace bytes of dwconv_linear_fwd (grad false) or dwconv_linear_grad."""
    if torch is None:
        _setup()
    return _size("dwconv_linear_workspace_size", int(bool(grad)), _types.get(dtype, -1),
                 _act(act), M, N, K)


def dwconv_linear_describe(product, dtype, M, N, K, aligned=True):
    """(kernel, ranges of the summed index) of LINEAR_Y, LINEAR_DX or LINEAR_DW;
    aligned: both operands' addresses and row strides are multiples of 16 bytes."""
    if torch is None:
        _setup()
    name, splits = ctypes.create_string_buffer(64), ctypes.c_int(0)
    _status(_library().dwconv_linear_describe(product, _types.get(dtype, -1), int(bool(aligned)),
                                              M, N, K, name, 64, ctypes.byref(splits)),
            "dwconv_linear_describe")
    return name.value.decode(), splits.value


def dwconv_linear_fwd(x, w, b, y, act="none", res=None, z=None, workspace=None, stream=None):
    """y = act(x w^T + b) + res; z receives the value before the activation."""
    code, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return dwconv_linear_fwd(x, w, b, y, act, res, z, workspace, st)
    px, ldx = _rows(x, "x", x)
    pw, ldw, N, K = _weights(w, x)
    shape = (*x.shape[:-1], N)
    pr, ldr = (None, 0) if res is None else _rows(res, "res", x, shape)
    pz, ldz = (None, 0) if z is None else _rows(z, "z", x, shape)
    _status(_library().dwconv_linear_fwd(
        px, ldx, pw, ldw, code, _dense(b, "b", x, _f32, (N,)), _act(act), pr, ldr,
        *_rows(y, "y", x, shape), pz, ldz, *_space(workspace, x), x.numel() // max(K, 1), N, K,
        st), "dwconv_linear_fwd")
    return y


def linear(x, w, b=None, act="none", res=None, save_z=False, stream=None):
    """y = act(x w^T + b) + res, or (y, z) with save_z, z the value before the
    activation.  x is (..., K), w (N, K), res and y (..., N), all of one type;
    b is (N,) float32."""
    _, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return linear(x, w, b, act, res, save_z, st)
    _, _, N, K = _weights(w, x)
    shape = (*x.shape[:-1], N)
    y = x.new_empty(shape)
    z = x.new_empty(shape) if save_z else None
    ws = _workspace(dwconv_linear_workspace_size(False, x.dtype, act, x.numel() // max(K, 1), N,
                                                 K), x)
    dwconv_linear_fwd(x, w, b, y, act, res, z, ws, st)
    return (y, z) if save_z else y


def dwconv_linear_grad(dy, x, w, dx, dw, db, z=None, workspace=None, act="none", stream=None):
    """Gradients of linear into dx, dw and db, each of which may be None."""
    code, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return dwconv_linear_grad(dy, x, w, dx, dw, db, z, workspace, act, st)
    pw, ldw, N, K = _weights(w, x)
    shape = (*x.shape[:-1], N)
    kind = _act(act)
    if kind != _pkg.ACT_NONE and z is None:
        raise ValueError("z is needed: the value before the activation that linear kept")
    none = (None, 0)
    _status(_library().dwconv_linear_grad(
        *_rows(dy, "dy", x, shape), *_rows(x, "x", x), pw, ldw, code, kind,
        *(none if kind == _pkg.ACT_NONE else _rows(z, "z", x, shape)),
        *(none if dx is None else _rows(dx, "dx", x, x.shape)),
        *(none if dw is None else _rows(dw, "dw", x, w.shape)), _dense(db, "db", x, _f32, (N,)),
        *_space(workspace, x), x.numel() // max(K, 1), N, K, st), "dwconv_linear_grad")
    return dx, dw, db


def linear_grad(dy, x, w, z=None, act="none", stream=None):
    """(dx, dw, db) of linear for the cotangent dy of y; z is what linear kept
    (save_z), needed unless act is none.  The residual's gradient is dy."""
    _, st, ctx = _start(x, stream)
    if ctx is not None:
        with ctx:
            return linear_grad(dy, x, w, z, act, st)
    _, _, N, K = _weights(w, x)
    dx = x.new_empty(x.shape)
    dw = x.new_empty((N, K))
    db = x.new_empty((N,), dtype=_f32)
    ws = _workspace(dwconv_linear_workspace_size(True, x.dtype, act, x.numel() // max(K, 1), N,
                                                 K), x)
    return dwconv_linear_grad(dy, x, w, dx, dw, db, z, ws, act, st)
