"""The sequence operators' C ABI and binding without a GPU: declarations, sizes
and refusals.  Fake device addresses; every call returns before any launch."""
import ctypes
import os
import re

import numpy as np
import pytest

import depthwise_convolution_amd as dw

from . import sequence_reference as ref

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "dwconv_seq.h")
A = 1 << 40          # fake addresses, 1 GiB apart
X, W, B, Y, Z, P, Q, R, V, U = (A + (k << 30) for k in range(10))


@pytest.fixture(scope="module")
def L():
    return dw.lib()


def _text():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_header_and_binding_agree(L):
    assert set(re.findall(r"\b(dwconv_\w+)\s*\(", _text())) == set(dw.SEQ_EXPORTS)
    for name in dw.SEQ_EXPORTS:
        assert hasattr(L, name) and callable(getattr(dw, name))
    d = dict(re.findall(r"#define\s+(DWCONV_\w+)\s+(\d+)", _text()))
    assert (int(d["DWCONV_T_F32"]), int(d["DWCONV_T_F16"]), int(d["DWCONV_T_BF16"])) == \
        (dw.T_F32, dw.T_F16, dw.T_BF16)
    assert int(d["DWCONV_CAUSAL_MAX_TAPS"]) == dw.CAUSAL_MAX_TAPS
    assert int(d["DWCONV_SCAN_RUN"]) == dw.SCAN_RUN


def _call(L, name, defaults, changes):
    a = dict(defaults, **changes)
    assert list(a) == list(defaults)
    return dw.STATUS[getattr(L, name)(*a.values())]


FWD = dict(x=X, ldx=64, type=2, w=W, wtype=0, b=B, act=3, init=P, y=Y, ldy=64, final=Q, seqs=2,
           tokens=10, offsets=None, C=64, K=4, stream=None)
CAUSAL_BAD = [
    (dict(x=None), "NULL_PTR"), (dict(w=None), "NULL_PTR"), (dict(y=None), "NULL_PTR"),
    (dict(type=3), "BAD_WTYPE"), (dict(type=-1), "BAD_WTYPE"), (dict(wtype=7), "BAD_WTYPE"),
    (dict(act=4), "BAD_EPILOGUE"), (dict(act=-1), "BAD_EPILOGUE"),
    (dict(seqs=0), "BAD_DIM"), (dict(tokens=-1), "BAD_DIM"), (dict(C=0), "BAD_DIM"),
    (dict(K=0), "BAD_DIM"), (dict(K=9), "BAD_DIM"), (dict(tokens=1 << 31), "BAD_DIM"),
    (dict(tokens=1 << 62), "BAD_DIM"), (dict(seqs=1 << 20, tokens=1 << 11), "BAD_DIM"),
    (dict(ldx=63), "ROW_STRIDE"), (dict(ldy=1), "ROW_STRIDE"), (dict(ldy=-64), "ROW_STRIDE"),
    (dict(ldx=1 << 40), "ROW_STRIDE"),
    (dict(x=X + 1), "MISALIGNED"), (dict(w=W + 2), "MISALIGNED"), (dict(b=B + 2), "MISALIGNED"),
    (dict(y=Y + 1), "MISALIGNED"), (dict(offsets=V + 2), "MISALIGNED"),
    (dict(y=X), "ALIAS"), (dict(y=X + 64), "ALIAS"), (dict(final=P), "ALIAS"),
    (dict(final=Y), "ALIAS"), (dict(final=X + 128), "ALIAS"), (dict(y=W), "ALIAS"),
    (dict(ldx=128, ldy=128, y=X + 2 * 63), "ALIAS"), (dict(ldx=128, ldy=96, y=X + 128), "ALIAS"),
]


@pytest.mark.parametrize("changes,code", CAUSAL_BAD)
def test_causal_fwd_refuses(L, changes, code):
    assert _call(L, "dwconv_causal_fwd", FWD, changes) == code


def test_causal_step_refuses(L):
    d = dict(x=X, ldx=64, type=1, w=W, wtype=1, b=B, act=0, state=P, y=Y, ldy=64, seqs=3, C=64,
             K=4, stream=None)
    for changes, code in [(dict(state=None), "NULL_PTR"), (dict(state=Y), "ALIAS"),
                          (dict(x=P), "ALIAS"), (dict(K=9), "BAD_DIM"), (dict(seqs=0), "BAD_DIM"),
                          (dict(ldy=10), "ROW_STRIDE"), (dict(type=5), "BAD_WTYPE"),
                          (dict(act=9), "BAD_EPILOGUE"), (dict(w=W + 1), "MISALIGNED")]:
        assert _call(L, "dwconv_causal_step", d, changes) == code, changes


def test_causal_grad_refuses(L):
    n = dw.dwconv_causal_grad_workspace_size(2, 10, False, 64, 4)
    d = dict(dy=Y, lddy=64, x=X, ldx=64, type=0, w=W, wtype=0, b=B, act=3, init=P, dfinal=Q,
             dx=Z, lddx=64, dw=R, db=R + 4096, dinit=V, ws=U, wsb=n, seqs=2, tokens=10,
             offsets=None, C=64, K=4, stream=None)
    assert n > 0
    for changes, code in [(dict(dy=None), "NULL_PTR"), (dict(dw=None), "NULL_PTR"),
                          (dict(dx=None), "NULL_PTR"), (dict(ws=None), "WORKSPACE"),
                          (dict(wsb=n - 1), "WORKSPACE"), (dict(ws=U + 4), "WORKSPACE"),
                          (dict(dx=Y), "ALIAS"), (dict(db=R + 4), "ALIAS"), (dict(ws=X), "ALIAS"),
                          (dict(dinit=P), "ALIAS"), (dict(lddx=3), "ROW_STRIDE"),
                          (dict(type=9), "BAD_WTYPE")]:
        assert _call(L, "dwconv_causal_grad", d, changes) == code, changes


SCAN = dict(x=X, ldx=64, r=P, ldr=128, i=P + 128, ldi=128, type=2, lam=W, scale=8.0, h0=B, y=Y,
            ldy=64, hT=Q, states=R, ws=U, wsb=1 << 20, seqs=2, tokens=10, offsets=None, C=64,
            stream=None)


def test_scan_fwd_refuses(L):
    for changes, code in [(dict(x=None), "NULL_PTR"), (dict(lam=None), "NULL_PTR"),
                          (dict(r=None), "NULL_PTR"), (dict(i=None), "NULL_PTR"),
                          (dict(y=None), "NULL_PTR"), (dict(type=4), "BAD_WTYPE"),
                          (dict(scale=0.0), "BAD_EPILOGUE"), (dict(scale=-1.0), "BAD_EPILOGUE"),
                          (dict(scale=float("nan")), "BAD_EPILOGUE"),
                          (dict(scale=float("inf")), "BAD_EPILOGUE"), (dict(C=0), "BAD_DIM"),
                          (dict(seqs=0), "BAD_DIM"), (dict(tokens=-5), "BAD_DIM"),
                          (dict(ldr=63), "ROW_STRIDE"), (dict(ldi=0), "ROW_STRIDE"),
                          (dict(hT=B), "ALIAS"), (dict(y=P), "ALIAS"), (dict(y=P + 128), "ALIAS"),
                          (dict(states=Q), "ALIAS"), (dict(hT=Q + 2), "MISALIGNED"),
                          (dict(r=P + 1), "MISALIGNED")]:
        assert _call(L, "dwconv_scan_fwd", SCAN, changes) == code, changes
    n = dw.dwconv_scan_workspace_size(False, 1, 100000, False, 64)     # runs are linked
    assert n > 0
    long = dict(seqs=1, tokens=100000)
    for changes in (dict(ws=None), dict(wsb=n - 1), dict(ws=U + 8)):
        assert _call(L, "dwconv_scan_fwd", SCAN, {**changes, **long}) == "WORKSPACE"


def test_scan_step_and_grad_refuse(L):
    d = dict(x=X, ldx=64, r=P, ldr=64, i=Q, ldi=64, type=0, lam=W, scale=8.0, h=B, y=Y, ldy=64,
             seqs=2, C=64, stream=None)
    for changes, code in [(dict(h=None), "NULL_PTR"), (dict(y=B), "ALIAS"), (dict(h=X), "ALIAS"),
                          (dict(scale=0.0), "BAD_EPILOGUE"), (dict(C=-1), "BAD_DIM"),
                          (dict(ldx=1), "ROW_STRIDE")]:
        assert _call(L, "dwconv_scan_step", d, changes) == code, changes
    n = dw.dwconv_scan_workspace_size(True, 2, 10, False, 64)
    d = dict(dy=Y, lddy=64, x=X, ldx=64, r=P, ldr=64, i=Q, ldi=64, type=1, lam=W, scale=8.0,
             states=B, dhT=R, dx=Z, lddx=64, dr=V, lddr=128, di=V + 128, lddi=128,
             dlam=R + (1 << 20), dh0=R + (2 << 20), ws=U, wsb=n, seqs=2, tokens=10, offsets=None,
             C=64, stream=None)
    for changes, code in [(dict(states=None), "NULL_PTR"), (dict(dlam=None), "NULL_PTR"),
                          (dict(dr=None), "NULL_PTR"), (dict(di=V + 126), "ALIAS"),
                          (dict(dx=X), "ALIAS"), (dict(dh0=R), "ALIAS"), (dict(ws=None), "WORKSPACE"),
                          (dict(wsb=n - 1), "WORKSPACE"), (dict(lddi=5), "ROW_STRIDE"),
                          (dict(scale=-2.0), "BAD_EPILOGUE")]:
        assert _call(L, "dwconv_scan_grad", d, changes) == code, changes


LINEAR = dict(x=X, ldx=32, w=W, ldw=32, type=2, b=B, act=3, res=P, ldres=48, y=Y, ldy=48, z=Z,
              ldz=48, ws=U, wsb=1 << 28, M=20, N=48, K=32, stream=None)


def test_linear_refuses(L):
    for changes, code in [(dict(x=None), "NULL_PTR"), (dict(w=None), "NULL_PTR"),
                          (dict(y=None), "NULL_PTR"), (dict(type=3), "BAD_WTYPE"),
                          (dict(act=4), "BAD_EPILOGUE"), (dict(M=-1), "BAD_DIM"),
                          (dict(M=1 << 31), "BAD_DIM"), (dict(N=0), "BAD_DIM"),
                          (dict(K=0), "BAD_DIM"), (dict(ldx=31), "ROW_STRIDE"),
                          (dict(ldw=8), "ROW_STRIDE"), (dict(ldy=47), "ROW_STRIDE"),
                          (dict(ldres=47), "ROW_STRIDE"), (dict(ldz=47), "ROW_STRIDE"),
                          (dict(y=P), "ALIAS"), (dict(z=Y), "ALIAS"), (dict(y=W), "ALIAS"),
                          (dict(y=B), "ALIAS"), (dict(b=B + 1), "MISALIGNED")]:
        assert _call(L, "dwconv_linear_fwd", LINEAR, changes) == code, changes
    n = dw.dwconv_linear_workspace_size(True, __import__("torch").bfloat16, "silu", 20, 48, 32)
    d = dict(dy=Y, lddy=48, x=X, ldx=32, w=W, ldw=32, type=2, act=3, z=Z, ldz=48, dx=P, lddx=32,
             dw=Q, lddw=32, db=R, ws=U, wsb=n, M=20, N=48, K=32, stream=None)
    for changes, code in [(dict(z=None), "NULL_PTR"), (dict(dy=None), "NULL_PTR"),
                          (dict(x=None), "NULL_PTR"), (dict(w=None), "NULL_PTR"),
                          (dict(dx=X), "ALIAS"), (dict(dw=P), "ALIAS"), (dict(wsb=n - 1), "WORKSPACE"),
                          (dict(ws=None), "WORKSPACE"), (dict(lddw=3), "ROW_STRIDE"),
                          (dict(type=-2), "BAD_WTYPE"), (dict(act=17), "BAD_EPILOGUE")]:
        assert _call(L, "dwconv_linear_grad", d, changes) == code, changes


def test_sizes(L):
    out = ctypes.c_longlong(0)
    assert dw.dwconv_scan_states_size(3, 100, False, 8) == (300 // dw.SCAN_RUN + 3) * 8
    assert dw.dwconv_scan_states_size(3, 0, True, 8) == 24
    # sequences that one workgroup scans at once have nothing to tell each other
    assert dw.dwconv_scan_workspace_size(False, 64, 128, False, 1024) == 0
    assert dw.dwconv_scan_workspace_size(False, 64, 129, False, 1024) > 0
    for name, args in (("dwconv_scan_states_size", (0, 5, 0, 8)),
                       ("dwconv_scan_workspace_size", (0, 1, -1, 0, 8)),
                       ("dwconv_causal_grad_workspace_size", (1, 5, 0, 8, 9)),
                       ("dwconv_linear_workspace_size", (0, 0, 0, 5, 0, 8))):
        assert dw.STATUS[getattr(L, name)(*args, ctypes.byref(out))] == "BAD_DIM"
        assert dw.STATUS[getattr(L, name)(*args, None)] == "NULL_PTR"


def test_binding_refuses_cpu_tensors_and_wrong_types():
    import torch
    x = torch.zeros(2, 3, 8)
    for call in (lambda: dw.causal_conv(x, torch.zeros(8, 4)),
                 lambda: dw.causal_conv_step(x[0], x, torch.zeros(8, 4)),
                 lambda: dw.gated_scan(x, x, x, torch.zeros(8)),
                 lambda: dw.gated_scan_step(x[0], x[0], x[0], torch.zeros(8), x[0]),
                 lambda: dw.linear(x, torch.zeros(4, 8)),
                 lambda: dw.linear_grad(x, x, torch.zeros(8, 8))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        dw.linear([1.0], torch.zeros(4, 8))


# ------------------------------- the reference's own gradients, by differences
def _check_gradient(loss, values, grads, names, rng):
    step = 1e-6
    for n in names:
        way = rng.standard_normal(values[n].shape)
        up, down = ({**values, n: values[n] + s * step * way} for s in (1, -1))
        change = (loss(up) - loss(down)) / (2 * step)
        assert abs(change - (grads[n] * way).sum()) <= 1e-6 * (np.abs(grads[n] * way).sum() + 1)


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(0)
    bounds = [(0, 3), (3, 3), (3, 14), (14, 15)]
    v = {n: rng.standard_normal((15, 5)) for n in ("x", "r", "i", "dy")}
    v |= {"lam": rng.standard_normal(5), "h0": rng.standard_normal((4, 5))}
    dhT = rng.standard_normal((4, 5))

    def loss(p):
        h, _, last, _ = ref.scan(p["x"], p["r"], p["i"], p["lam"], 2.0, bounds, p["h0"])
        return (h * v["dy"]).sum() + (last * dhT).sum()

    g = ref.scan_grad(v["dy"], v["x"], v["r"], v["i"], v["lam"], 2.0, bounds, v["h0"], dhT)
    names = ("x", "r", "i", "lam", "h0")
    _check_gradient(loss, v, {n: g["d" + n][0] for n in names}, names, rng)

    v |= {"w": rng.standard_normal((5, 4)), "b": rng.standard_normal(5),
          "init": rng.standard_normal((4, 3, 5))}
    dfinal = rng.standard_normal((4, 3, 5))

    def loss(p):
        z, _, last = ref.conv(p["x"], p["w"], p["b"], bounds, p["init"])
        return (ref.act(z, "silu") * v["dy"]).sum() + (last * dfinal).sum()

    g = ref.conv_grad(v["dy"], v["x"], v["w"], v["b"], bounds, v["init"], dfinal, "silu")
    names = ("x", "w", "b", "init")
    _check_gradient(loss, v, {n: g["d" + n][0] for n in names}, names, rng)
