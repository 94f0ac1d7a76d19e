"""Linear attention where nothing but the store of a result rounds (tests/mixing_exact.py):
every result equal to the exact one, rounded once."""
import numpy as np
import pytest

import depthwise_convolution_amd as dw

from . import mixing_exact as exact
from . import mixing_reference as ref
from .sequence_reference import bounds_of
from .test_gpu_mixing import DTYPES, _back, _gpu, _near, _offsets, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def _same(got, want, dtype, what):
    got, want = _back(got).reshape(want.shape), exact.rounded(want, dtype)
    bad = got != want
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} differ, first at "
                           f"{np.argwhere(bad)[0].tolist()}: {got[bad][0]} for {want[bad][0]}")


CASES = [
    # (lengths, H, KV, Dk, Dv): chunks that are whole and cut, segments, shared heads, odd widths
    ([64], 1, 1, 64, 64), ([1, 0, 63, 200], 2, 1, 64, 64), ([300], 2, 2, 40, 24),
    ([130, 67], 2, 2, 33, 17), ([150], 1, 1, 128, 128), ([90, 40], 1, 1, 160, 72),
    ([300], 4, 2, 16, 80),
    # many sequences that begin and end next to where the rows are cut
    ([63, 129, 1, 64, 65, 128, 1, 190, 0, 2, 66, 64, 64, 130, 62], 2, 1, 32, 24),
]


def _inputs(torch, case, dtype):     # noqa: F811
    lengths, H, KV, Dk, Dv = case
    rng = np.random.default_rng(len(lengths) * 1000 + Dk)
    rows, S = sum(lengths), len(lengths)
    r = dict(q=exact.whole(rng, (rows, H, Dk), 15), k=exact.whole(rng, (rows, KV, Dk), 15),
             v=exact.whole(rng, (rows, KV, Dv), 7), dy=exact.whole(rng, (rows, H, Dv), 15),
             h0=exact.whole(rng, (S, H, Dk, Dv), 4000),
             dhT=exact.whole(rng, (S, H, Dk, Dv), 4000, 2.0 ** -6))
    g = {n: _gpu(torch, t, "float32" if n in ("h0", "dhT") else dtype) for n, t in r.items()}
    for n in r:
        assert np.array_equal(_back(g[n]), r[n])
    logs = np.array([0.0, -np.inf, 0.0, 0.0][:H])
    g["log_decay"], g["off"] = _gpu(torch, logs), _gpu(torch, _offsets(lengths), "int32")
    return g, r, logs, bounds_of(_offsets(lengths))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_nothing_is_lost(torch, case, dtype):    # noqa: F811
    """The forward and every gradient, heads that forget nothing and all."""
    print(f"\n[case] exact attention {CASES[case]} {dtype}", flush=True)
    g, r, logs, bounds = _inputs(torch, CASES[case], dtype)
    scale = 2.0 ** -6
    args = r["q"], r["k"], r["v"]
    top = exact.majorants(*args, r["dy"], logs, scale, bounds, r["h0"], r["dhT"])
    for name, t in top.items():         # all sums are whole numbers of 2^-6 (hT: of 1)
        assert t.max(initial=0.0) < 2.0 ** (24 if name == "hT" else 18), name
    y, hT = dw.linear_attention(g["q"], g["k"], g["v"], g["log_decay"], h0=g["h0"],
                                offsets=g["off"], scale=scale)
    grads = dw.linear_attention_grad(g["dy"], g["q"], g["k"], g["v"], g["log_decay"], h0=g["h0"],
                                     dhT=g["dhT"], offsets=g["off"], scale=scale)
    torch.cuda.synchronize()
    want, state = ref.attention(*args, logs, scale, bounds, r["h0"])
    _same(y, want, dtype, "y")
    _same(hT, state, "float32", "hT")
    want = ref.attention_grad(r["dy"], *args, logs, scale, bounds, r["h0"], r["dhT"])
    for name, t in zip(("dq", "dk", "dv", "dh0"), grads):
        _same(t, want[name], "float32" if name == "dh0" else dtype, name)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("large", [20000.0, 60000.0])
def test_large_float16_values_leave_their_neighbours_exact(torch, large, D):    # noqa: F811
    """One value above 2^14 among columns around 2^-7: their states, and what later tokens
    read of them, keep every bit; and scores above 2^14 among small ones."""
    rng = np.random.default_rng(5)
    n = 200
    q, k = (exact.whole(rng, (n, 1, D), 15) for _ in range(2))
    v = exact.whole(rng, (n, 1, D), 7, 2.0 ** -10)
    v[5, 0, 3] = v[100, 0, D - 1] = large
    g, off, scale = np.zeros(1), [(0, n)], 2.0 ** -10
    want, state = ref.attention(q, k, v, g, scale, off, None)
    small = [c for c in range(D) if c not in (3, D - 1)]
    big, bs = ref.attention(*(np.abs(t) for t in (q, k, v)), g, scale, off, None)
    # whole numbers of 2^-20 and of 2^-10
    assert big[:, :, small].max() < 2.0 ** 4 and bs[:, :, :, small].max() < 2.0 ** 14
    args = [_gpu(torch, t[None], "float16") for t in (q, k, v)]
    y, hT = dw.linear_attention(*args, _gpu(torch, g), scale=scale)
    _same(hT[..., small], state[..., small], "float32", "hT")
    # the large ones themselves pass 2^18, with steps of 2^-10: 28 bits, of which float32
    # holds 24, so that each sum may round
    _near(hT, state, ref.attention_tol(bs, 0, n, "float32", 0.0, True), "all of hT")
    _same(y[..., small], want[..., small], "float16", "y")
    # scores: one query of 2^13 times the others
    q[70] *= 2.0 ** 10
    v[5, 0, 3] = v[100, 0, D - 1] = 0.0
    want, _ = ref.attention(q, k, v, g, scale * 2.0 ** 6, off, None)
    args = [_gpu(torch, t[None], "float16") for t in (q, k, v)]
    y, _ = dw.linear_attention(*args, _gpu(torch, g), scale=scale * 2.0 ** 6)
    _same(y, want, "float16", "y of large scores")


def test_float16_beside_a_large_state(torch):   # noqa: F811
    """Values and scores far below the state that they are added to: scaling them up does
    not take the state beyond float32."""
    D, n = 64, 130
    rng = np.random.default_rng(6)
    g, one = _gpu(torch, np.zeros(1)), np.ones((1, n, 1, D))
    # a state of 2^116 or 0, to which each token's product adds 2^-20
    h0 = exact.whole(rng, (1, 1, D, D), 100, 2.0 ** 110)
    q, k, v = (_gpu(torch, one * x, "float16") for x in (1.0, 1.0, 2.0 ** -20))
    _, hT = dw.linear_attention(q, k, v, g, h0=_gpu(torch, h0), scale=2.0 ** -120)
    _same(hT, (h0 + n * 2.0 ** -20).astype(np.float32).astype(np.float64), "float32", "hT")
    # and its cotangent, where the scale makes what is added 2^-130: the state, 2^27 at
    # most, has room for a factor of 2^72, so that 2^-25 of that is lost of a token
    dhT = exact.whole(rng, (1, 1, D, D), 100, 2.0 ** 20)
    dh0 = dw.linear_attention_grad(v, q, k, v, g, h0=_gpu(torch, h0), dhT=_gpu(torch, dhT),
                                   scale=2.0 ** -110)[3]
    _near(dh0, dhT + n * 2.0 ** -130, 2.0 ** -24 * np.abs(dhT) + n * 2.0 ** (-25 - 72), "dh0")
    # results of a large state beside scores of 2^-122: 7 * 64 * 2^6 in each
    q, k, v = (_gpu(torch, one * x, "float16") for x in (7.0, 2.0 ** -11, 1.0))
    h0 = np.full((1, 1, D, D), 2.0 ** 126)
    y, _ = dw.linear_attention(q, k, v, g, h0=_gpu(torch, h0), scale=2.0 ** -120)
    _same(y, np.full((1, n, 1, D), 28672.0), "float16", "y")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", [3, 6, 7])
def test_gradients_that_are_left_out(torch, case, dtype):   # noqa: F811
    """Every choice among dq, dk, dv and dh0, in sequences that are cut: the states of one
    walk serve another only where both are wanted."""
    print(f"\n[case] some gradients {CASES[case]} {dtype}", flush=True)
    g, r, logs, bounds = _inputs(torch, CASES[case], dtype)
    scale = 2.0 ** -6
    want = ref.attention_grad(r["dy"], r["q"], r["k"], r["v"], logs, scale, bounds, r["h0"],
                              r["dhT"])
    lengths, H, KV, Dk, Dv = CASES[case]
    n = dw.dwconv_attention_workspace_size(True, g["q"].dtype, len(lengths), sum(lengths), True, H,
                                           KV, Dk, Dv)
    for chosen in range(16):
        space = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None
        out = [torch.full_like(g[x], float("nan")) if chosen >> b & 1 else None
               for b, x in enumerate(("q", "k", "v", "h0"))]
        dw.dwconv_attention_grad(g["dy"], g["q"], g["k"], g["v"], g["log_decay"], *out,
                                 workspace=space, scale=scale, h0=g["h0"], dhT=g["dhT"],
                                 offsets=g["off"])
        for name, t in zip(("dq", "dk", "dv", "dh0"), out):
            if t is not None:
                _same(t, want[name], "float32" if name == "dh0" else dtype, (name, chosen))


# ------------------------------------------------------ float16 with any decay
DECAYS = [
    # (lengths, H, KV, Dk, Dv)
    ([200], 4, 4, 8, 8), ([64, 1, 0, 129], 4, 2, 16, 24), ([70, 300], 4, 1, 33, 17),
    ([150], 4, 4, 64, 64), ([130], 4, 2, 96, 80), ([100], 4, 4, 160, 40),
]


def decay_inputs(case):
    """float64 arrays of numbers that float16 holds."""
    lengths, H, KV, Dk, Dv = DECAYS[case]
    rng = np.random.default_rng(70 + case)

    def some(*shape):
        return rng.standard_normal(shape).astype(np.float16).astype(np.float64)

    rows, S = sum(lengths), len(lengths)
    r = dict(q=some(rows, H, Dk), k=some(rows, KV, Dk), v=some(rows, KV, Dv),
             dy=some(rows, H, Dv), h0=some(S, H, Dk, Dv), dhT=some(S, H, Dk, Dv))
    r["log_decay"] = np.array([-0.02, -1.0, -8.0, 0.0]).astype(np.float32).astype(np.float64)
    r["bounds"] = bounds_of(_offsets(lengths))
    return r, _offsets(lengths), Dk ** -0.5


@pytest.mark.parametrize("case", range(len(DECAYS)))
def test_float16_element_by_element(torch, case):     # noqa: F811
    """The forward and the gradients within what each element's own terms allow."""
    lengths, H, KV, Dk, Dv = DECAYS[case]
    print(f"\n[case] float16 attention {DECAYS[case]}", flush=True)
    r, offsets, scale = decay_inputs(case)
    g = {n: _gpu(torch, r[n], "float16") for n in ("q", "k", "v", "dy")}
    for n in ("h0", "dhT", "log_decay"):
        g[n] = _gpu(torch, r[n])
    off = _gpu(torch, offsets, "int32")
    y, _ = dw.linear_attention(g["q"], g["k"], g["v"], g["log_decay"], h0=g["h0"], offsets=off,
                               scale=scale)
    grads = dw.linear_attention_grad(g["dy"], g["q"], g["k"], g["v"], g["log_decay"], h0=g["h0"],
                                     dhT=g["dhT"], offsets=off, scale=scale)
    torch.cuda.synchronize()
    got = dict(zip(("dq", "dk", "dv"), grads), y=y)
    for name, (want, tol) in exact.float16_bounds(r, scale).items():
        _near(got[name], want, ref.store_tol(want, tol, "float16"), name)
