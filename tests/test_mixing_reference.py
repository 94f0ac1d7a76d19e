"""The float64 references of the mixing operators against finite differences."""
import numpy as np

from . import mixing_reference as ref


def _differences(f, x, step=1e-6):
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + step
        hi = f()
        x[i] = keep - step
        out[i] = (hi - f()) / (2 * step)
        x[i] = keep
    return out


def test_attention_gradients_are_differences():
    rng = np.random.default_rng(0)
    bounds = [(0, 3), (3, 3), (3, 8)]
    q, k, v = (rng.standard_normal(s) for s in ((8, 4, 3), (8, 2, 3), (8, 2, 2)))
    h0, dy = rng.standard_normal((3, 4, 3, 2)), rng.standard_normal((8, 4, 2))
    dhT, g = rng.standard_normal((3, 4, 3, 2)), np.array([-0.1, 0.3, -np.inf, -2.0])

    def loss():
        y, hT = ref.attention(q, k, v, g, 0.6, bounds, h0)
        return (y * dy).sum() + (hT * dhT).sum()

    grads = ref.attention_grad(dy, q, k, v, g, 0.6, bounds, h0, dhT)
    for name, x in (("dq", q), ("dk", k), ("dv", v), ("dh0", h0)):
        assert np.allclose(grads[name], _differences(loss, x), atol=1e-7), name


def test_norm_gradients_are_differences():
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((2, 3, 6)), rng.standard_normal((2, 3, 6))
    w, b = rng.standard_normal(6), rng.standard_normal(6)

    def loss():
        return (ref.Norm(x, 2, w, b, 1e-3, "silu").forward()[0] * dy).sum()

    grads = ref.Norm(x, 2, w, b, 1e-3, "silu").gradient(dy)
    for name, t in (("dx", x), ("dw", w), ("db", b)):
        assert np.allclose(grads[name][0], _differences(loss, t), atol=1e-7), name


def test_quantize_is_the_nearest():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((20, 50)) * 10.0 ** rng.integers(-30, 30, (20, 1))
    q, s = ref.quantize(x)
    off = np.abs(x / s.astype(np.float64)[:, None] - q)
    assert (off <= 0.5 + 1e-5).all() and (np.abs(q).max(1) == 127).all()
