"""The float64 device forms against the token-by-token ones, on the CPU."""
import numpy as np
import torch

from . import sequence_gpu64 as dev
from . import sequence_reference as ref

OFFSETS = [0, 0, 1, 4, 4, 40, 47, 47]


def _t(a):
    return torch.from_numpy(a)


def _same(got, want):
    assert np.allclose(got.numpy(), want, rtol=1e-11, atol=1e-13)


def test_conv():
    rng = np.random.default_rng(0)
    n, C, K, S = OFFSETS[-1], 5, 4, len(OFFSETS) - 1
    x, dy = rng.standard_normal((2, n, C))
    w, b, init = rng.standard_normal((C, K)), rng.standard_normal(C), rng.standard_normal(
        (S, K - 1, C))
    bounds, rows = ref.bounds_of(OFFSETS), dev.Rows(OFFSETS, "cpu")
    for carried in (None, init):
        z, _, final = ref.conv(x, w, b, bounds, carried)
        it = None if carried is None else _t(carried)
        got = dev.conv(_t(x), _t(w), _t(b), rows, it)
        _same(got, z)
        _same(dev.conv_final(_t(x), K, rows, it), final)
        want = ref.conv_grad(dy, x, w, b, bounds, carried, None, "silu")
        dz = _t(dy) * dev.slope(got, "silu")
        for name, t in zip(("dx", "dw", "db"), dev.conv_grad(dz, _t(x), _t(w), rows, it)):
            _same(t, want[name][0])


def test_scan():
    rng = np.random.default_rng(1)
    n, C, S = OFFSETS[-1], 5, len(OFFSETS) - 1
    x, r, i, dy = rng.standard_normal((4, n, C)) * 2
    lam, h0, dhT = rng.standard_normal(C) * 3, *rng.standard_normal((2, S, C))
    bounds, rows = ref.bounds_of(OFFSETS), dev.Rows(OFFSETS, "cpu")
    for start, end in ((None, None), (h0, dhT)):
        ts, te = (None if v is None else _t(v) for v in (start, end))
        s = dev.Scan(_t(x), _t(r), _t(i), _t(lam), 8.0, rows, ts)
        h, _, last, _ = ref.scan(x, r, i, lam, 8.0, bounds, start)
        _same(s.h, h)
        _same(s.last()[0], last)
        want = ref.scan_grad(dy, x, r, i, lam, 8.0, bounds, start, end)
        for name, (v, tol) in s.grad(_t(dy), te).items():
            _same(v, want[name][0])
            assert bool((tol >= 0).all())
