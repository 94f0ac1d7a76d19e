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

T_F32, T_F16, T_BF16 = 0, 1, 2
CAUSAL_MAX_TAPS = 8          # DWCONV_CAUSAL_MAX_TAPS
SCAN_RUN = 8                # DWCONV_SCAN_RUN

SEQ_EXPORTS = ("dwconv_causal_fwd", "dwconv_causal_step", "dwconv_causal_grad_workspace_size",
               "dwconv_causal_grad", "dwconv_scan_states_size", "dwconv_scan_workspace_size",
               "dwconv_scan_fwd", "dwconv_scan_step", "dwconv_scan_grad",
               "dwconv_linear_workspace_size", "dwconv_linear_fwd", "dwconv_linear_grad")

__all__ = ["causal_conv", "causal_conv_step", "causal_conv_grad", "gated_scan",
           "gated_scan_step", "gated_scan_grad", "linear", "linear_grad", "T_F32", "T_F16",
           "T_BF16", "CAUSAL_MAX_TAPS", "SCAN_RUN", "SEQ_EXPORTS", *SEQ_EXPORTS]


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
    L.dwconv_linear_fwd.argtypes = [*row * 2, i, vp, i, *row * 3, vp, ll, ll, i, i, vp]
    L.dwconv_linear_grad.argtypes = [*row * 3, i, i, *row * 3, vp, vp, ll, ll, i, i, vp]
    for name in SEQ_EXPORTS:
        getattr(L, name).restype = i


# ---------------------------------------------------------------- marshalling
_pkg = None
_types = None


def _setup():
    global _pkg, _types
    import torch

    import depthwise_convolution_amd as pkg
    _types = {torch.float32: T_F32, torch.float16: T_F16, torch.bfloat16: T_BF16}
    _pkg = pkg
    return pkg


def _library():
    return (_pkg or _setup()).lib()


def _type(t, name="x"):
    if _types is None:
        _setup()
    code = _types.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} has dtype {t.dtype}, expected float32, float16 or bfloat16")
    return code


def _gpu(t, name, like=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")
    if like is not None and t.device != like.device:
        raise ValueError("all tensors must be on the same device")


def _rows(t, name, shape=None, like=None):
    """(address, row stride) of a tensor whose rows are its last axis."""
    _gpu(t, name, like)
    if like is not None and t.dtype != like.dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {like.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    width = t.shape[-1]
    if t.is_contiguous():
        return t.data_ptr(), width
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


def _dense(t, name, dtype, shape, like):
    """Address of a dense tensor (None: NULL)."""
    if t is None:
        return None
    _gpu(t, name, like)
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _batch(x, offsets):
    """(sequences, tokens, offsets' address) of a dense or packed batch."""
    import torch
    _gpu(x, "x")
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


def _filter(w, x):
    _gpu(w, "w", x)
    if w.dim() != 2 or w.shape[0] != x.shape[-1] or not w.is_contiguous():
        raise ValueError("w must be a contiguous (C, taps) tensor")
    return w.data_ptr(), _type(w, "w"), w.shape[1]


class _Handle(int):
    """A hipStream_t that a call here has already made its tensors' stream."""


class _Place:
    """Where a call runs: `handle` is its hipStream_t.  Within the block the
    tensors' device and the stream are the current ones, so what is allocated
    belongs to the stream."""

    __slots__ = ("handle", "entered")

    def __init__(self, t, stream):
        import torch
        self.entered = None
        if type(stream) is _Handle:
            self.handle = stream
            return
        _gpu(t, "x")
        if stream is None:
            if t.device.index != torch.cuda.current_device():
                self.entered = torch.cuda.device(t.device)
            self.handle = _Handle(torch.cuda.current_stream(t.device).cuda_stream)
            return
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=t.device)
        self.handle = _Handle(stream.cuda_stream)
        self.entered = torch.cuda.stream(stream)

    def __enter__(self):
        if self.entered is not None:
            self.entered.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.entered is not None:
            self.entered.__exit__(*exc)


def _status(st, what):
    if st != 0:
        raise _pkg.DwconvError(st, what)


def _size(what, *args):
    out = ctypes.c_longlong(0)
    _status(getattr(_library(), what)(*args, ctypes.byref(out)), what)
    return out.value


def _workspace(nbytes, like):
    import torch
    return torch.empty(nbytes, dtype=torch.uint8, device=like.device) if nbytes else None


def _ws_args(ws):
    if ws is None:
        return None, 0
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor")
    return ws.data_ptr(), ws.numel() * ws.element_size()


# ------------------------------------------- causal depthwise convolution
def dwconv_causal_fwd(x, w, b, y, act="none", init=None, final=None, offsets=None, stream=None):
    """y = act(causal filter w of x, plus b); final receives the rows to carry."""
    import torch
    with _Place(x, stream) as st:
        seqs, tokens, off = _batch(x, offsets)
        C = x.shape[-1]
        px, ldx = _rows(x, "x")
        pw, wt, K = _filter(w, x)
        py, ldy = _rows(y, "y", x.shape, x)
        carried = (seqs, K - 1, C)
        _status(_library().dwconv_causal_fwd(
            px, ldx, _type(x), pw, wt, _dense(b, "b", torch.float32, (C,), x),
            _pkg._act_code(act), _dense(init, "init", x.dtype, carried, x), py, ldy,
            _dense(final, "final", x.dtype, carried, x), seqs, tokens, off, C, K, st),
            "dwconv_causal_fwd")
    return y


def causal_conv(x, w, b=None, act="none", init=None, offsets=None, stream=None):
    """(y, final): y = act(b + causal filter w of x), and the taps - 1 rows of
    each sequence that a continuation passes as init.

    w is (C, taps) of any of the types, b (C,) float32, init and final
    (sequences, taps - 1, C) of x's type, the oldest row first."""
    import torch
    with _Place(x, stream) as st:
        seqs, _, _ = _batch(x, offsets)
        _, _, K = _filter(w, x)
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        final = torch.empty((seqs, K - 1, x.shape[-1]), dtype=x.dtype, device=x.device)
        dwconv_causal_fwd(x, w, b, y, act, init, final, offsets, st)
    return y, final


def dwconv_causal_step(x, w, b, state, y, act="none", stream=None):
    """One token for each sequence; state (sequences, taps - 1, C) in place."""
    import torch
    with _Place(x, stream) as st:
        if x.dim() != 2:
            raise ValueError("x must be (sequences, C)")
        seqs, C = x.shape
        px, ldx = _rows(x, "x")
        pw, wt, K = _filter(w, x)
        py, ldy = _rows(y, "y", x.shape, x)
        _status(_library().dwconv_causal_step(
            px, ldx, _type(x), pw, wt, _dense(b, "b", torch.float32, (C,), x),
            _pkg._act_code(act), _dense(state, "state", x.dtype, (seqs, K - 1, C), x), py, ldy,
            seqs, C, K, st), "dwconv_causal_step")
    return y


def causal_conv_step(x, state, w, b=None, act="none", stream=None):
    """y (sequences, C) for one token of each sequence; state is updated in place."""
    import torch
    with _Place(x, stream) as st:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        return dwconv_causal_step(x, w, b, state, y, act, st)


def dwconv_causal_grad_workspace_size(seqs, tokens, packed, C, K):
    """Workspace bytes of dwconv_causal_grad (tokens: per sequence, or in all when packed)."""
    return _size("dwconv_causal_grad_workspace_size", seqs, tokens, int(bool(packed)), C, K)


def dwconv_causal_grad(dy, x, w, b, dx, dw, db, workspace, act="none", init=None, dfinal=None,
                       dinit=None, offsets=None, stream=None):
    """Gradients of causal_conv into dx, dw, db (or None) and dinit (or None)."""
    import torch
    with _Place(x, stream) as st:
        seqs, tokens, off = _batch(x, offsets)
        C = x.shape[-1]
        px, ldx = _rows(x, "x")
        pdy, lddy = _rows(dy, "dy", x.shape, x)
        pdx, lddx = _rows(dx, "dx", x.shape, x)
        pw, wt, K = _filter(w, x)
        carried, f32 = (seqs, K - 1, C), torch.float32
        if dw is None:
            raise TypeError("dw must be a torch.Tensor")
        _status(_library().dwconv_causal_grad(
            pdy, lddy, px, ldx, _type(x), pw, wt, _dense(b, "b", f32, (C,), x),
            _pkg._act_code(act), _dense(init, "init", x.dtype, carried, x),
            _dense(dfinal, "dfinal", x.dtype, carried, x), pdx, lddx,
            _dense(dw, "dw", f32, (C, K), x), _dense(db, "db", f32, (C,), x),
            _dense(dinit, "dinit", x.dtype, carried, x), *_ws_args(workspace), seqs, tokens, off,
            C, K, st), "dwconv_causal_grad")
    return dx, dw, db, dinit


def causal_conv_grad(dy, x, w, b=None, act="none", init=None, dfinal=None, offsets=None,
                     stream=None):
    """(dx, dw, db, dinit) of causal_conv for the cotangents dy of y and dfinal
    (or None) of final.  dw (C, taps) and db (C,) are float32; dinit is None
    unless init is given."""
    import torch
    with _Place(x, stream) as st:
        seqs, tokens, off = _batch(x, offsets)
        _, _, K = _filter(w, x)
        C, f32, dev = x.shape[-1], torch.float32, x.device
        dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
        dw = torch.empty((C, K), dtype=f32, device=dev)
        db = torch.empty((C,), dtype=f32, device=dev)
        dinit = None if init is None else torch.empty((seqs, K - 1, C), dtype=x.dtype, device=dev)
        ws = _workspace(dwconv_causal_grad_workspace_size(seqs, tokens, off is not None, C, K), x)
        return dwconv_causal_grad(dy, x, w, b, dx, dw, db, ws, act, init, dfinal, dinit, offsets,
                                  st)


# ------------------------------------------------- gated linear recurrence
def dwconv_scan_states_size(seqs, tokens, packed, C):
    """Floats that dwconv_scan_fwd keeps for the gradient."""
    return _size("dwconv_scan_states_size", seqs, tokens, int(bool(packed)), C)


def dwconv_scan_workspace_size(grad, seqs, tokens, packed, C):
    """Workspace bytes of dwconv_scan_fwd (grad false) or dwconv_scan_grad."""
    return _size("dwconv_scan_workspace_size", int(bool(grad)), seqs, tokens, int(bool(packed)),
                 C)


def dwconv_scan_fwd(x, r, i, lam, y, hT=None, states=None, workspace=None, scale=8.0, h0=None,
                    offsets=None, stream=None):
    """y = the states of the recurrence; hT the last ones; states for the gradient."""
    import torch
    with _Place(x, stream) as st:
        seqs, tokens, off = _batch(x, offsets)
        C, f32 = x.shape[-1], torch.float32
        px, ldx = _rows(x, "x")
        pr, ldr = _rows(r, "r", x.shape, x)
        pi, ldi = _rows(i, "i", x.shape, x)
        py, ldy = _rows(y, "y", x.shape, x)
        if lam is None:
            raise TypeError("lam must be a torch.Tensor")
        if states is not None:
            _dense(states, "states", f32,
                   (dwconv_scan_states_size(seqs, tokens, off is not None, C),), x)
        _status(_library().dwconv_scan_fwd(
            px, ldx, pr, ldr, pi, ldi, _type(x), _dense(lam, "lam", f32, (C,), x), scale,
            _dense(h0, "h0", f32, (seqs, C), x), py, ldy, _dense(hT, "hT", f32, (seqs, C), x),
            None if states is None else states.data_ptr(), *_ws_args(workspace), seqs, tokens,
            off, C, st), "dwconv_scan_fwd")
    return y


def gated_scan(x, r, i, lam, h0=None, offsets=None, scale=8.0, save_states=False, stream=None):
    """(y, hT), or (y, hT, states) with save_states: the gated recurrence

        h = a * h + sqrt(1 - a^2) * sigmoid(i) * x,
        log a = -scale * softplus(lam) * sigmoid(r)

    per channel, y its states in x's type, hT (sequences, C) float32 the last
    ones, states what gated_scan_grad needs.  r and i are the gates before
    their sigmoid, shaped as x; lam is (C,), h0 (sequences, C), both float32."""
    import torch
    with _Place(x, stream) as st:
        seqs, tokens, off = _batch(x, offsets)
        C, f32, dev = x.shape[-1], torch.float32, x.device
        packed = off is not None
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
        hT = torch.empty((seqs, C), dtype=f32, device=dev)
        states = None
        if save_states:
            states = torch.empty((dwconv_scan_states_size(seqs, tokens, packed, C),), dtype=f32,
                                 device=dev)
        ws = _workspace(dwconv_scan_workspace_size(False, seqs, tokens, packed, C), x)
        dwconv_scan_fwd(x, r, i, lam, y, hT, states, ws, scale, h0, offsets, st)
    return (y, hT, states) if save_states else (y, hT)


def dwconv_scan_step(x, r, i, lam, h, y, scale=8.0, stream=None):
    """One token for each sequence; h (sequences, C) float32 in place."""
    import torch
    with _Place(x, stream) as st:
        if x.dim() != 2:
            raise ValueError("x must be (sequences, C)")
        seqs, C = x.shape
        px, ldx = _rows(x, "x")
        pr, ldr = _rows(r, "r", x.shape, x)
        pi, ldi = _rows(i, "i", x.shape, x)
        py, ldy = _rows(y, "y", x.shape, x)
        _status(_library().dwconv_scan_step(
            px, ldx, pr, ldr, pi, ldi, _type(x), _dense(lam, "lam", torch.float32, (C,), x),
            scale, _dense(h, "h", torch.float32, (seqs, C), x), py, ldy, seqs, C, st),
            "dwconv_scan_step")
    return y


def gated_scan_step(x, r, i, lam, h, scale=8.0, stream=None):
    """y (sequences, C) for one token of each sequence; h is updated in place."""
    import torch
    with _Place(x, stream) as st:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        return dwconv_scan_step(x, r, i, lam, h, y, scale, st)


def dwconv_scan_grad(dy, x, r, i, lam, states, dx, dr, di, dlam, dh0=None, workspace=None,
                     scale=8.0, dhT=None, offsets=None, stream=None):
    """Gradients of gated_scan into dx, dr, di, dlam and dh0 (or None)."""
    import torch
    with _Place(x, stream) as st:
        seqs, tokens, off = _batch(x, offsets)
        C, f32 = x.shape[-1], torch.float32
        named = (("dy", dy), ("x", x), ("r", r), ("i", i), ("dx", dx), ("dr", dr), ("di", di))
        p = [v for name, t in named for v in _rows(t, name, x.shape, x)]
        if lam is None or dlam is None:
            raise TypeError("lam and dlam must be torch.Tensors")
        ps = _dense(states, "states", f32,
                    (dwconv_scan_states_size(seqs, tokens, off is not None, C),), x)
        _status(_library().dwconv_scan_grad(
            *p[:8], _type(x), _dense(lam, "lam", f32, (C,), x), scale, ps,
            _dense(dhT, "dhT", f32, (seqs, C), x), *p[8:], _dense(dlam, "dlam", f32, (C,), x),
            _dense(dh0, "dh0", f32, (seqs, C), x), *_ws_args(workspace), seqs, tokens, off, C,
            st), "dwconv_scan_grad")
    return dx, dr, di, dlam, dh0


def gated_scan_grad(dy, x, r, i, lam, states, dhT=None, offsets=None, scale=8.0, stream=None):
    """(dx, dr, di, dlam, dh0) of gated_scan for the cotangents dy of y and dhT
    (or None) of hT; states are those that gated_scan kept.  dlam (C,) and dh0
    (sequences, C) are float32."""
    import torch
    with _Place(x, stream) as st:
        seqs, tokens, off = _batch(x, offsets)
        C, f32, dev = x.shape[-1], torch.float32, x.device
        dx, dr, di = (torch.empty(x.shape, dtype=x.dtype, device=dev) for _ in range(3))
        dlam = torch.empty((C,), dtype=f32, device=dev)
        dh0 = torch.empty((seqs, C), dtype=f32, device=dev)
        ws = _workspace(dwconv_scan_workspace_size(True, seqs, tokens, off is not None, C), x)
        return dwconv_scan_grad(dy, x, r, i, lam, states, dx, dr, di, dlam, dh0, ws, scale, dhT,
                                offsets, st)


# --------------------------------- matrix product with bias, activation, residual
def dwconv_linear_workspace_size(grad, dtype, act, M, N, K):
    """Workspace bytes of dwconv_linear_fwd (grad false) or dwconv_linear_grad."""
    if _types is None:
        _setup()
    return _size("dwconv_linear_workspace_size", int(bool(grad)), _types.get(dtype, -1),
                 _pkg._act_code(act), M, N, K)


def _weights(w, x):
    pw, ldw = _rows(w, "w", None, x)
    if w.dim() != 2 or w.shape[1] != x.shape[-1]:
        raise ValueError("w must be (N, K) with K the last axis of x")
    return pw, ldw, w.shape[0], w.shape[1]


def dwconv_linear_fwd(x, w, b, y, act="none", res=None, z=None, workspace=None, stream=None):
    """y = act(x w^T + b) + res; z receives the value before the activation."""
    import torch
    with _Place(x, stream) as st:
        px, ldx = _rows(x, "x")
        pw, ldw, N, K = _weights(w, x)
        shape = (*x.shape[:-1], N)
        M = x.numel() // max(K, 1)
        py, ldy = _rows(y, "y", shape, x)
        pr, ldr = (None, 0) if res is None else _rows(res, "res", shape, x)
        pz, ldz = (None, 0) if z is None else _rows(z, "z", shape, x)
        _status(_library().dwconv_linear_fwd(
            px, ldx, pw, ldw, _type(x), _dense(b, "b", torch.float32, (N,), x),
            _pkg._act_code(act), pr, ldr, py, ldy, pz, ldz, *_ws_args(workspace), M, N, K, st),
            "dwconv_linear_fwd")
    return y


def linear(x, w, b=None, act="none", res=None, save_z=False, stream=None):
    """y = act(x w^T + b) + res, or (y, z) with save_z, z the value before the
    activation.  x is (..., K), w (N, K), res and y (..., N), all of one type;
    b is (N,) float32."""
    import torch
    with _Place(x, stream) as st:
        _, _, N, K = _weights(w, x)
        shape = (*x.shape[:-1], N)
        y = torch.empty(shape, dtype=x.dtype, device=x.device)
        z = torch.empty(shape, dtype=x.dtype, device=x.device) if save_z else None
        ws = _workspace(dwconv_linear_workspace_size(False, x.dtype, act, x.numel() // max(K, 1), N, K),
                        x)
        dwconv_linear_fwd(x, w, b, y, act, res, z, ws, st)
    return (y, z) if save_z else y


def dwconv_linear_grad(dy, x, w, dx, dw, db, z=None, workspace=None, act="none", stream=None):
    """Gradients of linear into dx, dw and db, each of which may be None."""
    import torch
    with _Place(x, stream) as st:
        px, ldx = _rows(x, "x")
        pw, ldw, N, K = _weights(w, x)
        shape = (*x.shape[:-1], N)
        M = x.numel() // max(K, 1)
        pdy, lddy = _rows(dy, "dy", shape, x)
        code = _pkg._act_code(act)
        if code != _pkg.ACT_NONE and z is None:
            raise ValueError("z is needed: the value before the activation that linear kept")
        pz, ldz = (None, 0) if z is None or code == _pkg.ACT_NONE else _rows(z, "z", shape, x)
        pdx, lddx = (None, 0) if dx is None else _rows(dx, "dx", x.shape, x)
        pdw, lddw = (None, 0) if dw is None else _rows(dw, "dw", w.shape, x)
        _status(_library().dwconv_linear_grad(
            pdy, lddy, px, ldx, pw, ldw, _type(x), code, pz, ldz, pdx, lddx, pdw, lddw,
            _dense(db, "db", torch.float32, (N,), x), *_ws_args(workspace), M, N, K, st),
            "dwconv_linear_grad")
    return dx, dw, db


def linear_grad(dy, x, w, z=None, act="none", stream=None):
    """(dx, dw, db) of linear for the cotangent dy of y; z is what linear kept
    (save_z), needed unless act is none.  The residual's gradient is dy."""
    import torch
    with _Place(x, stream) as st:
        _, _, N, K = _weights(w, x)
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dw = torch.empty((N, K), dtype=w.dtype, device=x.device)
        db = torch.empty((N,), dtype=torch.float32, device=x.device)
        ws = _workspace(dwconv_linear_workspace_size(True, x.dtype, act, x.numel() // max(K, 1), N, K), x)
        return dwconv_linear_grad(dy, x, w, dx, dw, db, z, ws, act, st)
