"""What the exact cases of linear attention tell apart, without a GPU: scores or a state
in one number of a 16-bit type, and a gradient that lacks a term, change their results."""
import numpy as np
import pytest

from . import mixing_exact as exact
from . import mixing_reference as ref
from .test_gpu_mixing_exact import DECAYS, decay_inputs


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_one_number_of_a_type_shows(dtype):
    rng = np.random.default_rng(1)
    q, k = (exact.whole(rng, (200, 1, 64), 15) for _ in range(2))
    v = exact.whole(rng, (200, 1, 64), 7)
    h0, scale = exact.whole(rng, (1, 64, 64), 4000), 2.0 ** -6
    want, state = ref.attention(q, k, v, np.zeros(1), scale, [(0, 200)], h0[None])
    P = exact.scores(q, k, scale, 0, 64)
    bits = 11 if dtype == "float16" else 8
    assert exact.holds(P, 16) and not exact.holds(P, bits)
    assert exact.holds(state, 16) and not exact.holds(state, bits)
    once = exact.rounded(want, dtype)
    for part in (slice(0, 64), slice(64, 200)):     # h0 alone, and what joins it
        got = exact.rounded(exact.one_number(q, k, v, h0, scale, dtype)[part], dtype)
        assert (got != once[part]).mean() > 0.05, part


def test_rounding():
    x = np.array([1.0, 1.00390625, 1.01171875, -3.0, 65519.0, 65520.0, 1 + 2.0 ** -8 + 2.0 ** -20])
    import torch
    for dtype in ("float16", "bfloat16"):
        want = torch.from_numpy(x).to(torch.float32).to(getattr(torch, dtype)).double().numpy()
        assert np.array_equal(exact.rounded(x, dtype), want)


def test_a_dropped_term_shows():
    rng = np.random.default_rng(2)
    q, k = (exact.whole(rng, (70, 1, 16), 15) for _ in range(2))
    v, dy = exact.whole(rng, (70, 1, 16), 7), exact.whole(rng, (70, 1, 16), 15)
    args = np.zeros(1), 2.0 ** -6, [(0, 70)], None, None
    want = ref.attention_grad(dy, q, k, v, *args)
    one = v.copy()
    one[3, 0, 5] = 0
    lost = ref.attention_grad(dy, q, k, one, *args)
    assert (exact.rounded(want["dq"], "float16")[3:] !=
            exact.rounded(lost["dq"], "float16")[3:]).mean() > 0.5


def _outside(got, want, tol):
    return np.abs(exact.rounded(got, "float16") - want) > ref.store_tol(want, tol, "float16")


@pytest.mark.parametrize("case", range(len(DECAYS)))
def test_the_float16_bounds_tell_mistakes_apart(case):
    """They hold for the exact results, rounded once, and not without one token's term."""
    r, _, scale = decay_inputs(case)
    bounds = exact.float16_bounds(r, scale)
    for name, (want, tol) in bounds.items():
        assert not _outside(want, want, tol).any(), name
        # what float16's range costs is small beside the rounding of a typical result
        floor = exact.float16_floors(r, scale)[name]
        assert np.median(floor) < 2.0 ** -13 * np.median(np.abs(want)), name
    t = r["bounds"][0][1] // 2
    for lost in ("k", "v", "q", "dy"):
        one = dict(r, **{lost: r[lost].copy()})
        one[lost][t, 0, 0] = 0.0
        got = exact.float16_bounds(one, scale)
        for name, (want, tol) in bounds.items():
            own = {"q": "dq", "k": "dk", "v": "dv"}.get(lost)
            if name != own and not (name == "y" and lost == "dy"):
                assert _outside(got[name][0], want, tol).any(), (lost, name)


def test_the_float16_bounds_tell_one_number_apart():
    r, _, scale = decay_inputs(0)
    want, tol = exact.float16_bounds(r, scale)["y"]
    head = 3            # the one that forgets nothing, whose scores are not decayed
    got = exact.one_number(r["q"][:, head:], r["k"][:, head:], r["v"][:, head:],
                           r["h0"][0, head:], scale, "float16")
    assert _outside(got, want[:, head:], tol[:, head:]).mean() > 0.01
