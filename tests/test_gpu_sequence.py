"""GPU parity of the sequence operators against float64 references.

Tolerances come from the number of float32 roundings on the way to each
result (tests/sequence_reference.py), never from what a run gave.  Inputs are
drawn in float64 and rounded to the tensors' type first, so the reference sees
the same values.
"""
import numpy as np
import pytest

import depthwise_convolution_amd as dw

from . import sequence_reference as ref

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "float16", "bfloat16"]
# sequences of a packed batch: of no token, of one, shorter than the filter,
# around the scan's run length, and longer
RAGGED = [0, 1, 0, 2, 3, 127, 128, 129, 1, 300, 0]


@pytest.fixture(scope="module")
def torch():
    import torch as t
    if not t.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    return t


def _dt(torch, name):
    return getattr(torch, name)


def _gpu(torch, a, dtype="float32"):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", _dt(torch, dtype))


def _back(t):
    return t.detach().double().cpu().numpy()


def _draw(torch, rng, shape, dtype, scale=1.0):
    """(GPU tensor, its values in float64)."""
    t = _gpu(torch, rng.standard_normal(shape) * scale, dtype)
    return t, _back(t)


def _near(got, want, tol, what):
    got = _back(got).reshape(want.shape)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst error / tolerance "
                           f"{np.nanmax(np.abs(got - want) / tol):.3g}")


def _offsets(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)


def _wide(torch, t, pad=5):
    """The same values as a column range of a wider tensor."""
    big = torch.full((*t.shape[:-1], t.shape[-1] + 2 * pad), float("nan"), dtype=t.dtype,
                     device=t.device)
    view = big[..., pad:pad + t.shape[-1]]
    view.copy_(t)
    return view


# ------------------------------------------- causal depthwise convolution
CONV_CASES = [
    # (lengths or (S, T), C, K, act, carry, strided)
    (RAGGED, 64, 4, "silu", True, False),
    (RAGGED, 67, 3, "none", False, True),
    ((3, 50), 131, 2, "silu", True, False),
    ((2, 33), 3, 4, "relu", False, False),
    ((1, 1), 8, 8, "none", True, False),
    ((2, 0), 16, 4, "none", True, False),
    ([0, 0, 0], 16, 4, "none", True, False),
    ((4, 70), 40, 1, "relu6", False, False),
    ((2, 40), 1, 5, "silu", True, True),
    ((5, 3), 24, 6, "none", True, False),
    ((1, 257), 520, 7, "silu", False, False),
]


def _conv_inputs(torch, case, dtype, seed, integers=False):
    layout, C, K, act, carry, strided = case
    rng = np.random.default_rng(seed)
    packed = isinstance(layout, list)
    offsets = _offsets(layout) if packed else _offsets([layout[1]] * layout[0])
    shape = (int(offsets[-1]), C) if packed else (*layout, C)
    S = len(offsets) - 1

    def draw(shape, dtype):
        if integers:        # small whole numbers: every sum is exact
            t = _gpu(torch, rng.integers(-3, 4, shape).astype(np.float64), dtype)
            return t, _back(t)
        return _draw(torch, rng, shape, dtype)

    x, xr = draw(shape, dtype)
    w, wr = draw((C, K), "float32" if dtype == "float32" or C % 2 else dtype)
    b, br = draw((C,), "float32")
    init, initr = draw((S, K - 1, C), dtype) if carry else (None, None)
    dy, dyr = draw(shape, dtype)
    dfinal, dfinalr = draw((S, K - 1, C), dtype) if carry else (None, None)
    if strided:
        x, dy = _wide(torch, x), _wide(torch, dy)
    off = torch.from_numpy(offsets).cuda() if packed else None
    return dict(x=x, w=w, b=b, init=init, dy=dy, dfinal=dfinal, off=off), dict(
        x=xr.reshape(-1, C), w=wr, b=br, init=initr, dy=dyr.reshape(-1, C), dfinal=dfinalr,
        bounds=ref.bounds_of(offsets))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(CONV_CASES)))
def test_causal_conv(torch, case, dtype):
    spec = CONV_CASES[case]
    K, act = spec[2], spec[3]
    print(f"\n[case] causal_conv {spec} {dtype}", flush=True)
    g, r = _conv_inputs(torch, spec, dtype, case)
    y, final = dw.causal_conv(g["x"], g["w"], g["b"], act=act, init=g["init"], offsets=g["off"])
    torch.cuda.synchronize()
    assert y.shape == g["x"].shape and y.dtype == g["x"].dtype
    z, big, wfinal = ref.conv(r["x"], r["w"], r["b"], r["bounds"], r["init"])
    tol = ref.act_tol(z, EPS_SUM(K) * big, act)
    want = ref.act(z, act)
    _near(y, want, ref.store_tol(want, tol, dtype), "y")
    assert np.array_equal(_back(final), wfinal)      # copies
    # no bias
    y2, _ = dw.causal_conv(g["x"], g["w"], None, act="none", init=g["init"], offsets=g["off"])
    z2, big2, _ = ref.conv(r["x"], r["w"], 0 * r["b"], r["bounds"], r["init"])
    _near(y2, z2, ref.store_tol(z2, EPS_SUM(K) * big2, dtype), "y without bias")


def EPS_SUM(n):
    """Relative to the majorant: n fused multiply-adds and the bias."""
    return (n + 2) * ref.EPS


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(CONV_CASES)))
def test_causal_conv_grad(torch, case, dtype):
    spec = CONV_CASES[case]
    K, act = spec[2], spec[3]
    print(f"\n[case] causal_conv_grad {spec} {dtype}", flush=True)
    # with a corner in the activation, z has to be exact to fall on the same side
    g, r = _conv_inputs(torch, spec, dtype, 100 + case, integers=act.startswith("relu"))
    dx, dW, db, dinit = dw.causal_conv_grad(g["dy"], g["x"], g["w"], g["b"], act=act,
                                            init=g["init"], dfinal=g["dfinal"],
                                            offsets=g["off"])
    torch.cuda.synchronize()
    want = ref.conv_grad(r["dy"], r["x"], r["w"], r["b"], r["bounds"], r["init"], r["dfinal"],
                         act)
    # dz: z's error through a second derivative of at most 0.5 where |z| is
    # moderate, the slope's own (16 + 2|z|) roundings
    _, zbig, _ = ref.conv(r["x"], r["w"], r["b"], r["bounds"], r["init"])
    zmax = np.abs(zbig).max() if zbig.size else 0.0
    rows = max(1, r["x"].shape[0])
    c = (24 + 4 * zmax + K + 0.5 * (K + 2) * zmax) * ref.EPS
    dyabs = np.abs(r["dy"])

    def tol(name, n):
        # the slope can be near 0 where its error is not: majorants with |dy|
        # in place of |dz| (slopes are at most 1.1)
        return (c + n * ref.EPS) * big[name] * 1.1 + 1e-30

    big = {k: v[1] for k, v in
           ref.conv_grad(dyabs, np.abs(r["x"]), np.abs(r["w"]), r["b"], r["bounds"],
                         None if r["init"] is None else np.abs(r["init"]),
                         None if r["dfinal"] is None else np.abs(r["dfinal"]), "none").items()}
    _near(dx, want["dx"][0], ref.store_tol(want["dx"][0], tol("dx", K), dtype), "dx")
    _near(dW, want["dw"][0], tol("dw", rows), "dw")
    _near(db, want["db"][0], tol("db", rows), "db")
    if g["init"] is None:
        assert dinit is None
    else:
        _near(dinit, want["dinit"][0], ref.store_tol(want["dinit"][0], tol("dinit", K), dtype),
              "dinit")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("S,C,K,act", [(1, 1, 4, "silu"), (7, 64, 4, "silu"), (3, 67, 1, "none"),
                                       (5, 129, 8, "relu"), (300, 20, 2, "relu6")])
def test_causal_conv_step_continues(torch, S, C, K, act, dtype):
    """Token by token from a prompt's carried rows equals one call over all."""
    print(f"\n[case] causal_conv_step {S} {C} {K} {act} {dtype}", flush=True)
    rng = np.random.default_rng(7)
    T, new = 5, 4
    x, xr = _draw(torch, rng, (S, T + new, C), dtype)
    w, wr = _draw(torch, rng, (C, K), "float32")
    b, br = _draw(torch, rng, (C,), "float32")
    whole, last = dw.causal_conv(x, w, b, act=act)
    y, state = dw.causal_conv(x[:, :T].contiguous(), w, b, act=act)
    assert torch.equal(y, whole[:, :T])
    for t in range(T, T + new):
        got = dw.causal_conv_step(x[:, t], state, w, b, act=act)    # rows of a wider tensor
        torch.cuda.synchronize()
        assert torch.equal(got, whole[:, t]), f"token {t}"
    assert torch.equal(state, last)


def test_causal_conv_keeps_sequences_apart(torch):
    """NaN and infinities in one sequence stay there."""
    lengths = [5, 3, 9, 0, 40]
    off = _offsets(lengths)
    rng = np.random.default_rng(3)
    x, _ = _draw(torch, rng, (int(off[-1]), 24), "float32")
    x[5:8] = float("nan")
    x[8 + 9 - 1] = float("inf")
    w, _ = _draw(torch, rng, (24, 4), "float32")
    dy, _ = _draw(torch, rng, tuple(x.shape), "float32")
    offsets = torch.from_numpy(off).cuda()
    y, final = dw.causal_conv(x, w, act="silu", offsets=offsets)
    dx, _, _, _ = dw.causal_conv_grad(dy, x, w, act="silu", offsets=offsets)
    torch.cuda.synchronize()
    for t in (y, dx):
        assert torch.isnan(t[5:8]).all()
        assert torch.isfinite(t[:5]).all() and torch.isfinite(t[17:]).all()
        assert torch.isfinite(t[8:13]).all()
    assert torch.isfinite(final[[0, 3, 4]]).all()


# ------------------------------------------------- gated linear recurrence
SCAN_CASES = [
    # (lengths or (S, T), C, carry, strided)
    (RAGGED, 64, True, False),
    (RAGGED, 70, False, True),
    ((2, 128), 64, True, False),
    ((1, 1), 4, True, False),
    ((3, 5), 3, True, False),
    ((2, 0), 8, True, False),
    ([0, 0], 8, True, False),
    ((1, 700), 1, True, True),
    ((1, 1500), 130, False, False),
    ((3, 2600), 66, True, False),           # runs looked back over more than once
    ([40] * 150 + [700], 5, True, False),   # more sequences than one search step sees
    ([1, 900, 0, 300, 2000, 5], 36, True, False),
]


def _scan_inputs(torch, case, dtype, seed):
    layout, C, carry, strided = case
    rng = np.random.default_rng(seed)
    packed = isinstance(layout, list)
    offsets = _offsets(layout) if packed else _offsets([layout[1]] * layout[0])
    shape = (int(offsets[-1]), C) if packed else (*layout, C)
    S = len(offsets) - 1
    g, r = {}, {"bounds": ref.bounds_of(offsets)}
    for name, sc in (("x", 1.0), ("r", 2.0), ("i", 2.0), ("dy", 1.0)):
        g[name], v = _draw(torch, rng, shape, dtype, sc)
        r[name] = v.reshape(-1, C)
        if strided:
            g[name] = _wide(torch, g[name])
    # memories from a few tokens to thousands, one channel that hardly decays
    decay = rng.uniform(0.2, 0.9995, C)
    lam = np.log(np.expm1(-np.log(decay) / 8.0))
    if C > 2:
        lam[1] = -30.0
    g["lam"] = _gpu(torch, lam)
    r["lam"] = _back(g["lam"])
    g["h0"], r["h0"] = _draw(torch, rng, (S, C), "float32") if carry else (None, None)
    g["dhT"], r["dhT"] = _draw(torch, rng, (S, C), "float32") if carry else (None, None)
    g["off"] = torch.from_numpy(offsets).cuda() if packed else None
    return g, r


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(SCAN_CASES)))
def test_gated_scan(torch, case, dtype):
    spec = SCAN_CASES[case]
    print(f"\n[case] gated_scan {spec} {dtype}", flush=True)
    g, r = _scan_inputs(torch, spec, dtype, case)
    y, hT = dw.gated_scan(g["x"], g["r"], g["i"], g["lam"], h0=g["h0"], offsets=g["off"])
    torch.cuda.synchronize()
    h, err, last, last_err = ref.scan(r["x"], r["r"], r["i"], r["lam"], 8.0, r["bounds"],
                                      r["h0"])
    _near(y, h, ref.store_tol(h, err, dtype), "y")
    _near(hT, last, ref.store_tol(last, last_err, "float32"), "hT")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(SCAN_CASES)))
def test_gated_scan_grad(torch, case, dtype):
    spec = SCAN_CASES[case]
    print(f"\n[case] gated_scan_grad {spec} {dtype}", flush=True)
    g, r = _scan_inputs(torch, spec, dtype, 50 + case)
    y, hT, states = dw.gated_scan(g["x"], g["r"], g["i"], g["lam"], h0=g["h0"],
                                  offsets=g["off"], save_states=True)
    got = dw.gated_scan_grad(g["dy"], g["x"], g["r"], g["i"], g["lam"], states, dhT=g["dhT"],
                             offsets=g["off"])
    torch.cuda.synchronize()
    want = ref.scan_grad(r["dy"], r["x"], r["r"], r["i"], r["lam"], 8.0, r["bounds"], r["h0"],
                         r["dhT"])
    # g and h each take up to (6 + 32 m) roundings a token on the way (see the
    # reference's scan; 40 covers m <= 1), the gates and products 128 more, and
    # dlam's sum one a token
    longest = max([hi - lo for lo, hi in r["bounds"]] + [1])
    rows = r["x"].shape[0]
    c = (128 + 2 * 40 * min(longest, 400)) * ref.EPS
    for name, t, kind in zip(("dx", "dr", "di", "dlam", "dh0"), got,
                             (dtype, dtype, dtype, "float32", "float32")):
        v, big = want[name]
        extra = rows * ref.EPS if name == "dlam" else 0.0
        _near(t, v, ref.store_tol(v, (c + extra) * big + 1e-30, kind), name)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("S,C", [(1, 1), (9, 64), (3, 67), (300, 6)])
def test_gated_scan_step_continues(torch, S, C, dtype):
    print(f"\n[case] gated_scan_step {S} {C} {dtype}", flush=True)
    T, new = 6, 3
    g, r = _scan_inputs(torch, ((S, T + new), C, True, False), dtype, 9)
    whole, last = dw.gated_scan(g["x"], g["r"], g["i"], g["lam"], h0=g["h0"])
    _, h = dw.gated_scan(*(g[n][:, :T].contiguous() for n in ("x", "r", "i")), g["lam"],
                         h0=g["h0"])
    hs, err, fin, fin_err = ref.scan(r["x"], r["r"], r["i"], r["lam"], 8.0, r["bounds"],
                                     r["h0"])
    hs, err = hs.reshape(S, -1, C), err.reshape(S, -1, C)
    for t in range(T, T + new):
        y = dw.gated_scan_step(*(g[n][:, t] for n in ("x", "r", "i")), g["lam"], h)
        torch.cuda.synchronize()
        _near(y, hs[:, t], ref.store_tol(hs[:, t], err[:, t], dtype), f"token {t}")
    _near(h, fin, ref.store_tol(fin, fin_err, "float32"), "state")


def test_gated_scan_shut_and_open_gates(torch):
    """Gates at the ends of their range: r = -inf keeps the state and takes
    nothing in, with finite gradients; i = -inf takes nothing in; large lam
    forgets everything."""
    S, T, C = 1, 140, 8
    rng = np.random.default_rng(5)
    x, xr = _draw(torch, rng, (S, T, C), "float32")
    r, i = torch.zeros_like(x), torch.zeros_like(x)
    lam = torch.zeros(C, device="cuda")
    h0 = torch.ones(S, C, device="cuda")
    r[..., 0] = -float("inf")
    r[..., 1] = -1e4
    i[..., 2] = -float("inf")
    i[..., 3] = float("inf")
    lam[4] = 1e4                # a = 0 at every token: h = sigmoid(i) x
    y, hT, states = dw.gated_scan(x, r, i, lam, h0=h0, save_states=True)
    dy = torch.ones_like(x)
    dx, dr, di, dlam, dh0 = dw.gated_scan_grad(dy, x, r, i, lam, states)
    torch.cuda.synchronize()
    assert torch.equal(y[..., :2], torch.ones_like(y[..., :2]))
    decay = 0.5 * 8.0 * np.log(2.0)
    assert np.allclose(_back(y[0, :, 2]), np.exp(-decay * np.arange(1, T + 1)), rtol=1e-4,
                       atol=1e-30)
    assert np.allclose(_back(y[0, :, 4]), 0.5 * xr[0, :, 4], rtol=1e-5)
    for t in (y, hT, dx, dr, di, dlam, dh0):
        assert torch.isfinite(t).all()
    assert (dx[..., :2] == 0).all() and (dr[..., :2] == 0).all() and (di[..., 2:4] == 0).all()
    assert torch.equal(dh0[0, :2], torch.full((2,), float(T), device="cuda"))


def test_gated_scan_keeps_sequences_apart(torch):
    lengths = [130, 40, 0, 300]
    off = torch.from_numpy(_offsets(lengths)).cuda()
    g, _ = _scan_inputs(torch, (lengths, 64, True, False), "float32", 2)
    g["x"][130:135] = float("nan")
    g["dy"][130:135] = float("inf")
    y, hT, states = dw.gated_scan(g["x"], g["r"], g["i"], g["lam"], h0=g["h0"], offsets=off,
                                  save_states=True)
    dx, dr, di, _, dh0 = dw.gated_scan_grad(g["dy"], g["x"], g["r"], g["i"], g["lam"], states,
                                            offsets=off)
    torch.cuda.synchronize()
    for t in (y, dx, dr, di):
        assert torch.isfinite(t[:130]).all() and torch.isfinite(t[170:]).all()
    assert torch.isnan(y[130:170]).all()
    assert torch.isfinite(hT[[0, 2, 3]]).all() and torch.isfinite(dh0[[0, 2, 3]]).all()


# --------------------------------- matrix product with bias, activation, residual
LINEAR_CASES = [
    # (M, N, K, act, bias, residual, strided)
    (1, 1, 1, "none", False, False, False),
    (1, 96, 64, "silu", True, True, False),
    (3, 130, 257, "relu", True, False, False),
    (8, 256, 512, "none", True, True, False),
    (17, 33, 70, "relu6", False, True, True),
    (64, 64, 64, "silu", True, False, False),
    (100, 200, 72, "none", False, False, False),
    (129, 257, 136, "silu", True, True, True),
    (300, 128, 1000, "relu", True, True, False),
    (513, 260, 40, "silu", False, True, False),
    (1000, 48, 7, "none", True, False, False),
    (256, 512, 1024, "silu", True, True, False),
    (31, 1024, 2048, "none", True, False, False),
    (0, 8, 8, "none", True, False, False),
    (20011, 70, 90, "silu", True, True, False),     # many ranges of rows in dw
    (520, 300, 64, "relu6", True, True, False),     # a tile's last columns by vectors
    (260, 515, 96, "silu", True, True, True),       # and by elements
]


def _linear_inputs(torch, case, dtype, seed):
    M, N, K, act, bias, res, strided = case
    rng = np.random.default_rng(seed)
    g, r = {}, {}
    for name, shape, sc in (("x", (M, K), 1.0), ("w", (N, K), K ** -0.5), ("res", (M, N), 1.0),
                            ("dy", (M, N), 1.0)):
        g[name], r[name] = _draw(torch, rng, shape, dtype, sc)
        if strided:
            g[name] = _wide(torch, g[name])
    g["b"], r["b"] = _draw(torch, rng, (N,), "float32")
    if not bias:
        g["b"] = r["b"] = None
    if not res:
        g["res"] = r["res"] = None
    return g, r


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(LINEAR_CASES)))
def test_linear(torch, case, dtype):
    spec = LINEAR_CASES[case]
    M, N, K, act = spec[:4]
    print(f"\n[case] linear {spec} {dtype}", flush=True)
    g, r = _linear_inputs(torch, spec, dtype, case)
    y, z = dw.linear(g["x"], g["w"], g["b"], act=act, res=g["res"], save_z=True)
    torch.cuda.synchronize()
    wz, big = ref.linear(r["x"], r["w"], r["b"])
    # K products and additions, twice a unit roundoff each in case the matrix
    # instructions truncate; float32 products to 4 units (three-way split)
    zerr = (2 * K + 12) * ref.EPS * big
    _near(z, wz, ref.store_tol(wz, zerr, dtype), "z")
    want = ref.act(wz, act)
    tol = ref.act_tol(wz, zerr, act)
    if r["res"] is not None:
        want = want + r["res"]
        tol = tol + ref.EPS * np.abs(want)
    _near(y, want, ref.store_tol(want, tol, dtype), "y")
    y2 = dw.linear(g["x"], g["w"], g["b"], act=act, res=g["res"])
    assert torch.equal(y, y2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(LINEAR_CASES)))
def test_linear_grad(torch, case, dtype):
    spec = LINEAR_CASES[case]
    M, N, K, act = spec[:4]
    print(f"\n[case] linear_grad {spec} {dtype}", flush=True)
    g, r = _linear_inputs(torch, spec, dtype, 70 + case)
    z = (g["x"].float() @ g["w"].float().t()).to(g["x"].dtype)
    dx, dW, db = dw.linear_grad(g["dy"], g["x"], g["w"], z=None if act == "none" else z, act=act)
    torch.cuda.synchronize()
    zr = _back(z)
    want = ref.linear_grad(r["dy"], r["x"], r["w"], zr, act)
    u = ref.ROUND[dtype] if act != "none" else 0.0      # dz is rounded to the type
    # the slope's error: (16 + 2|z|) roundings, of at most 1.1 |dy|
    slope_err = (16 + 2 * (np.abs(zr).max() if zr.size else 0)) * ref.EPS if act == "silu" \
        else ref.EPS
    ady = 1.1 * np.abs(r["dy"])
    big = {"dx": ady @ np.abs(r["w"]), "dw": ady.T @ np.abs(r["x"]), "db": ady.sum(0)}
    small = ref.TINY[dtype]
    extra = {"dx": small * np.abs(r["w"]).sum(0), "dw": small * np.abs(r["x"]).sum(0)}
    for name, t, n in (("dx", dx, N), ("dw", dW, M)):
        v, b = want[name]
        tol = ((2 * n + 12) * ref.EPS + u) * b * (1 + u) + slope_err * big[name] + extra[name]
        _near(t, v, ref.store_tol(v, tol, dtype), name)
    v, b = want["db"]
    _near(db, v, (M + 4) * ref.EPS * b + slope_err * big["db"] + 1e-30, "db")


def test_linear_into_column_ranges(torch):
    """Two products into the halves of one tensor, nothing else written."""
    rng = np.random.default_rng(4)
    for dtype in DTYPES:
        x, xr = _draw(torch, rng, (37, 48), dtype)
        w, wr = _draw(torch, rng, (2, 24, 48), dtype)
        out = torch.full((37, 60), 7.0, dtype=x.dtype, device="cuda")
        ws = None
        n = dw.dwconv_linear_workspace_size(False, x.dtype, "none", 37, 24, 48)
        if n:
            ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        dw.dwconv_linear_fwd(x, w[0], None, out[:, 2:26], workspace=ws)
        dw.dwconv_linear_fwd(x, w[1], None, out[:, 30:54], workspace=ws)
        torch.cuda.synchronize()
        for k, lo in enumerate((2, 30)):
            z, big = ref.linear(xr, wr[k], None)
            _near(out[:, lo:lo + 24], z, ref.store_tol(z, 108 * ref.EPS * big, dtype), "half")
        rest = torch.cat([out[:, :2], out[:, 26:30], out[:, 54:]], 1)
        assert (rest == 7.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_odd_extents_in_aligned_rows(torch, dtype):
    """Views whose rows start on 16 bytes but end on an odd element, in the order of
    every product: the last element of the last row counts."""
    rng = np.random.default_rng(6)
    M, N, K = 67, 129, 73
    g, r = {}, {}
    for name, shape in (("x", (M, K)), ("w", (N, K)), ("dy", (M, N))):
        t, r[name] = _draw(torch, rng, shape, dtype)
        big = torch.full((shape[0], 160), float("nan"), dtype=t.dtype, device="cuda")
        g[name] = big[:, :shape[1]]
        g[name].copy_(t)
    y = dw.linear(g["x"], g["w"])
    dx, dW, db = dw.linear_grad(g["dy"], g["x"], g["w"])
    torch.cuda.synchronize()
    z, big = ref.linear(r["x"], r["w"], None)
    _near(y, z, ref.store_tol(z, (2 * K + 12) * ref.EPS * big, dtype), "y")
    want = ref.linear_grad(r["dy"], r["x"], r["w"], None, "none")
    for name, t, n in (("dx", dx, N), ("dw", dW, M)):
        v, b = want[name]
        _near(t, v, ref.store_tol(v, (2 * n + 12) * ref.EPS * b, dtype), name)
    v, b = want["db"]
    _near(db, v, (M + 4) * ref.EPS * b + 1e-30, "db")


def test_linear_passes_infinities_and_nan(torch):
    """A row of x with NaN or infinity reaches its own row of y only, and
    finite float32 values beyond the 16-bit types' precision stay finite."""
    for dtype in DTYPES:
        for M in (5, 200):
            x = torch.ones(M, 64, dtype=_dt(torch, dtype), device="cuda")
            x[1, 3] = float("inf")
            x[2, 60] = float("nan")
            x[4, 0] = -float("inf")
            w = torch.full((72, 64), 0.5, dtype=x.dtype, device="cuda")
            y = dw.linear(x, w)
            torch.cuda.synchronize()
            assert torch.isinf(y[1]).all() and (y[1] > 0).all(), dtype
            assert torch.isnan(y[2]).all() and (y[4] < 0).all() and torch.isinf(y[4]).all()
            rest = torch.cat([y[:1], y[3:4], y[5:]])
            assert (rest == 32.0).all()
    big = torch.full((4, 16), 2.0 ** 60, device="cuda")
    assert (dw.linear(big, big) == 16 * 2.0 ** 120).all()
    top = torch.full((4, 1), 3.4e38, device="cuda")
    one = torch.ones(4, 1, device="cuda")
    assert torch.equal(dw.linear(top, one), top.expand(4, 4))


# ------------------------------------------------------------ all of them
def test_same_bits_twice_and_on_another_stream(torch):
    g, _ = _scan_inputs(torch, SCAN_CASES[-1], "bfloat16", 1)
    c, _ = _conv_inputs(torch, CONV_CASES[0], "float16", 1)
    l, _ = _linear_inputs(torch, LINEAR_CASES[7], "bfloat16", 1)

    def everything(stream):
        out = list(dw.gated_scan(g["x"], g["r"], g["i"], g["lam"], h0=g["h0"], offsets=g["off"],
                                 save_states=True, stream=stream))
        out[2:] = dw.gated_scan_grad(g["dy"], g["x"], g["r"], g["i"], g["lam"], out[2],
                                     dhT=g["dhT"], offsets=g["off"], stream=stream)
        out += dw.causal_conv(c["x"], c["w"], c["b"], act="silu", init=c["init"],
                              offsets=c["off"], stream=stream)
        out += dw.causal_conv_grad(c["dy"], c["x"], c["w"], c["b"], act="silu", init=c["init"],
                                   dfinal=c["dfinal"], offsets=c["off"], stream=stream)
        out += dw.linear(l["x"], l["w"], l["b"], act="silu", res=l["res"], save_z=True,
                         stream=stream)
        out += dw.linear_grad(l["dy"], l["x"], l["w"], z=out[-1], act="silu", stream=stream)
        return out

    first = everything(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        again = everything(stream)
        # memory of the side stream's workspaces, taken again by the current one
        noise = [torch.full((1 << 16,), 3.0, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        assert len(noise) == 8
        for k, (a, b) in enumerate(zip(first, again)):
            assert torch.equal(a, b), f"output {k} on {stream}"


def test_graph_replays_match_eager(torch):
    """A recurrent block's forward and gradients captured once and replayed,
    with eager work between the replays."""
    g, _ = _scan_inputs(torch, ((2, 300), 64, True, False), "bfloat16", 1)
    l, _ = _linear_inputs(torch, (600, 64, 64, "silu", True, True, False), "bfloat16", 1)
    wc = torch.randn(64, 4, device="cuda") / 2

    def step():
        u, z = dw.linear(l["x"], l["w"], l["b"], act="silu", res=l["res"], save_z=True)
        v, _ = dw.causal_conv(u.view(2, 300, 64), wc, act="silu")
        y, hT, states = dw.gated_scan(v, g["r"], g["i"], g["lam"], h0=g["h0"], save_states=True)
        dv, dr, di, dlam, _ = dw.gated_scan_grad(g["dy"], v, g["r"], g["i"], g["lam"], states)
        du, dwc, _, _ = dw.causal_conv_grad(dv, u.view(2, 300, 64), wc, act="silu")
        dx, dW, db = dw.linear_grad(du.view(600, 64), l["x"], l["w"], z=z, act="silu")
        return [y, hT, dr, di, dlam, dwc, dx, dW, db]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        want = [t.clone() for t in step()]
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for rep in range(4):
        for t in got:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), f"replay {rep}: output {k}"
        with torch.cuda.stream(side):
            step()
        side.synchronize()


def test_gradients_against_differences(torch):
    """Along a random direction of all inputs, the GPU's gradients predict the
    change of a float64 forward (central difference; its own error is below
    1e-6 of the change here, the float32 gradients' below 1e-5)."""
    rng = np.random.default_rng(12)
    # recurrence
    g, r = _scan_inputs(torch, ([3, 0, 150, 20], 16, True, False), "float32", 12)
    _, _, states = dw.gated_scan(g["x"], g["r"], g["i"], g["lam"], h0=g["h0"], offsets=g["off"],
                                 save_states=True)
    grads = dw.gated_scan_grad(g["dy"], g["x"], g["r"], g["i"], g["lam"], states, dhT=g["dhT"],
                               offsets=g["off"])
    names = ("x", "r", "i", "lam", "h0")

    def loss(v):
        h, _, last, _ = ref.scan(v["x"], v["r"], v["i"], v["lam"], 8.0, r["bounds"], v["h0"])
        return (h * r["dy"]).sum() + (last * r["dhT"]).sum()

    _along(rng, names, r, grads, loss)
    # filter
    c, q = _conv_inputs(torch, ([4, 0, 1, 60], 16, 4, "silu", True, False), "float32", 12)
    grads = dw.causal_conv_grad(c["dy"], c["x"], c["w"], c["b"], act="silu", init=c["init"],
                                dfinal=c["dfinal"], offsets=c["off"])

    def loss(v):
        z, _, last = ref.conv(v["x"], v["w"], v["b"], q["bounds"], v["init"])
        return (ref.act(z, "silu") * q["dy"]).sum() + (last * q["dfinal"]).sum()

    _along(rng, ("x", "w", "b", "init"), q, grads, loss)
    # product
    l, p = _linear_inputs(torch, (40, 24, 50, "silu", True, False, False), "float32", 12)
    _, z = dw.linear(l["x"], l["w"], l["b"], act="silu", save_z=True)
    grads = dw.linear_grad(l["dy"], l["x"], l["w"], z=z, act="silu")

    def loss(v):
        z, _ = ref.linear(v["x"], v["w"], v["b"])
        return (ref.act(z, "silu") * p["dy"]).sum()

    _along(rng, ("x", "w", "b"), p, grads, loss)


def _along(rng, names, values, grads, loss):
    step = 1e-5
    way = {n: rng.standard_normal(values[n].shape) for n in names}
    up, down = ({**values, **{n: values[n] + s * step * way[n] for n in names}} for s in (1, -1))
    change = (loss(up) - loss(down)) / (2 * step)
    parts = [_back(t).reshape(way[n].shape) * way[n] for n, t in zip(names, grads)]
    told = sum(p.sum() for p in parts)
    assert abs(told - change) <= 1.1e-5 * sum(np.abs(p).sum() for p in parts), (told, change)
