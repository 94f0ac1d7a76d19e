"""GPU parity of the gated recurrence where chains have more runs than the chip
holds at once, and where its gates are nearly open or shut, with bounds on the
errors that follow the steps (tests/sequence_gpu64.py).
"""
import numpy as np
import pytest

import depthwise_convolution_amd as dw

from .test_gpu_causal_large import _cuts

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "float16", "bfloat16"]


@pytest.fixture(scope="module")
def torch():
    import torch as t
    if not t.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    return t


@pytest.fixture(scope="module")
def ref():
    from . import sequence_gpu64
    return sequence_gpu64


@pytest.fixture(autouse=True)
def _free():
    yield
    import torch as t
    if t.cuda.is_available():
        t.cuda.empty_cache()


# ------------------------------------------------- gated linear recurrence
def _scan_inputs(torch, rng, layout, seqs, C, dtype, carry, gates=2.0):
    if seqs is None:
        seqs, offsets = layout[0], np.arange(layout[0] + 1) * layout[1]
        shape, off = (*layout, C), None
    else:
        offsets = _cuts(rng, layout, seqs, 6)
        shape, off = (layout, C), torch.from_numpy(offsets).cuda()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(rng.integers(1 << 30)))

    def draw(*shape, std=1.0, kind=dtype):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(getattr(torch, kind))

    g = {"x": draw(*shape), "r": draw(*shape, std=gates), "i": draw(*shape, std=gates),
         "dy": draw(*shape), "off": off}
    # memories from a few tokens to thousands, one channel that hardly decays
    decay = rng.uniform(0.2, 0.9995, C)
    lam = np.log(np.expm1(-np.log(decay) / 8.0))
    lam[C // 2] = -30.0
    g["lam"] = torch.from_numpy(lam).float().cuda()
    g["h0"] = draw(seqs, C, kind="float32") if carry else None
    g["dhT"] = draw(seqs, C, kind="float32") if carry else None
    return g, offsets


def _check_scan(torch, ref, g, offsets, dtype):
    C = g["x"].shape[-1]
    y, hT, states = dw.gated_scan(g["x"], g["r"], g["i"], g["lam"], h0=g["h0"], offsets=g["off"],
                                  save_states=True)
    got = dw.gated_scan_grad(g["dy"], g["x"], g["r"], g["i"], g["lam"], states, dhT=g["dhT"],
                             offsets=g["off"])
    torch.cuda.synchronize()
    flat = {n: g[n].double().reshape(-1, C) for n in ("x", "r", "i", "dy")}
    wide = {n: None if g[n] is None else g[n].double() for n in ("h0", "dhT")}
    s = ref.Scan(flat["x"], flat["r"], flat["i"], g["lam"].double(), 8.0, ref.Rows(offsets),
                 wide["h0"])
    ref.near(y, s.h, ref.store_tol(s.h, s.err, dtype), "y")
    last, err = s.last()
    ref.near(hT, last, ref.store_tol(last, err, "float32"), "hT")
    want = s.grad(flat["dy"], wide["dhT"])
    for name, t, kind in zip(("dx", "dr", "di", "dlam", "dh0"), got,
                             (dtype, dtype, dtype, "float32", "float32")):
        v, tol = want[name]
        ref.near(t, v, ref.store_tol(v, tol + 1e-30, kind), name)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout,seqs,C,carry", [
    ((3, 20000), None, 512, True),      # 3768 workgroups: the chip holds 768 or fewer
    (50021, 29, 640, False),            # 4190
    (30000, 3001, 320, True),           # 16175, most of a sequence of a few tokens
])
def test_gated_scan_large(torch, ref, layout, seqs, C, carry, dtype):
    print(f"\n[case] large gated_scan {layout} {seqs} {C} {carry} {dtype}", flush=True)
    rng = np.random.default_rng(11)
    g, offsets = _scan_inputs(torch, rng, layout, seqs, C, dtype, carry)
    _check_scan(torch, ref, g, offsets, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_scan_of_nearly_open_and_shut_gates(torch, ref, dtype):
    """Gates of 6 to 18 either way: 1 - sigma is as small as e^-18, and keeps its
    digits in dr and di."""
    print(f"\n[case] gated_scan gates of 6 to 18 {dtype}", flush=True)
    rng = np.random.default_rng(5)
    g, offsets = _scan_inputs(torch, rng, (6, 333), None, 72, dtype, True)
    for n in ("r", "i"):
        v = rng.uniform(6.0, 18.0, tuple(g["x"].shape)) * rng.choice([-1.0, 1.0], g["x"].shape)
        g[n] = torch.from_numpy(v).to("cuda", g["x"].dtype)
    _check_scan(torch, ref, g, offsets, dtype)


def test_decays_of_long_memories(torch):
    """sqrt(1 - a^2) of channels that decay by 8 e^-4 to 8 e^-85 a token, by one step
    from zero with open gates.  In roundings of 2^-24: the exponential 3, the
    logarithm's polynomial 3, the scale 1, u's polynomial and product 2.6, 2 m - m^2
    1, of which the root leaves half, and its own 2."""
    lam = torch.linspace(-85.0, -4.0, 4001, device="cuda")
    x = torch.ones(1, 4001, device="cuda")
    gate = torch.full_like(x, float("inf"))
    h = torch.zeros_like(x)
    dw.gated_scan_step(x, gate, gate, lam, h)
    y, hT = dw.gated_scan(x[None], gate[None], gate[None], lam)
    torch.cuda.synchronize()
    rate = 8.0 * torch.log1p(torch.exp(lam.double()))
    want = torch.sqrt(-torch.expm1(-2.0 * rate))
    for t in (h[0], hT[0], y[0, 0]):
        off = (t.double() - want).abs() / want * 2.0 ** 24
        assert float(off.max()) <= 0.5 * (3 + 3 + 1 + 2.6 + 1) + 2, float(off.max())
