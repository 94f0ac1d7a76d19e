"""The mixing operators in float64 numpy, and error bounds.

Shares no code with the GPU path.  Linear attention goes token by token; beside
each result stands its majorant, the same sums over absolute values, from
which the tests take their tolerances (unit roundoff of float32: 2^-24).
"""
import numpy as np

from .sequence_reference import EPS, ROUND, act, act_tol, slope, store_tol  # noqa: F401


# ---------------------------- linear attention with a decay for each head
def decay(log_decay):
    with np.errstate(over="ignore"):
        return np.exp(np.minimum(log_decay, 0.0))


def attention(q, k, v, log_decay, scale, bounds, h0):
    """(y, hT); q (rows, H, Dk), k (rows, KV, Dk), v (rows, KV, Dv)."""
    H, KV, Dk, Dv = q.shape[1], k.shape[1], k.shape[2], v.shape[2]
    head = np.arange(H) // (H // KV)
    a = decay(log_decay)[:, None, None]
    y, hT = np.zeros((len(q), H, Dv)), np.zeros((len(bounds), H, Dk, Dv))
    for s, (lo, hi) in enumerate(bounds):
        S = np.zeros((H, Dk, Dv)) if h0 is None else h0[s].copy()
        for t in range(lo, hi):
            S = a * S + k[t, head][:, :, None] * v[t, head][:, None, :]
            y[t] = scale * np.einsum("hk,hkv->hv", q[t], S)
        hT[s] = S
    return y, hT


def attention_grad(dy, q, k, v, log_decay, scale, bounds, h0, dhT):
    """dict of dq, dk, dv, dh0."""
    H, KV, Dk, Dv = q.shape[1], k.shape[1], k.shape[2], v.shape[2]
    head = np.arange(H) // (H // KV)
    a = decay(log_decay)[:, None, None]
    out = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v),
           "dh0": np.zeros((len(bounds), H, Dk, Dv))}
    for s, (lo, hi) in enumerate(bounds):
        S = np.zeros((H, Dk, Dv)) if h0 is None else h0[s].copy()
        for t in range(lo, hi):
            S = a * S + k[t, head][:, :, None] * v[t, head][:, None, :]
            out["dq"][t] = scale * np.einsum("hkv,hv->hk", S, dy[t])
        G = np.zeros((H, Dk, Dv)) if dhT is None else dhT[s].copy()
        for t in range(hi - 1, lo - 1, -1):
            G = G + scale * q[t][:, :, None] * dy[t][:, None, :]
            np.add.at(out["dk"][t], head, np.einsum("hkv,hv->hk", G, v[t, head]))
            np.add.at(out["dv"][t], head, np.einsum("hkv,hk->hv", G, k[t, head]))
            G = a * G
        out["dh0"][s] = G
    return out


def attention_tol(big, sums, tokens, dtype, floor=0.0, states=False):
    """Error of a result of linear attention before its store, from its majorant
    `big`; `sums`: the widths that its products are summed over.

    16-bit types: each of a result's terms passes one operand rounded to the type
    (a score, or the state that a chunk starts from), half a step; `floor` is what
    float16 loses of values far below the largest.  float32: sums of `sums` and of
    the 64 tokens of a chunk (twice a unit each, in case the matrix instructions
    truncate), two roundings for each of at least 32 tokens that a state passes
    through, one for each of the segments' links, and the powers of the decay,
    whose exponent of at most 88 is rounded: 1.25 * 88 and 18 more for what stands
    beside them."""
    c = 2 * (sums + 64) + 4 * (tokens // 32 + 2) + 128
    r = 0.0 if dtype == "float32" or states else ROUND[dtype] * (1 + ROUND[dtype])
    # the parts that a state is built from hold 22 bits and more: 2^-22 = 4 units
    return (c + 4) * EPS * big + r * big + floor


# ------------------------------------- group normalisation with an activation
def _parts(x, groups):
    """(N, groups, P, C / groups) of channels-last x."""
    N, C = x.shape[0], x.shape[-1]
    return x.reshape(N, -1, groups, C // groups).transpose(0, 2, 1, 3)


def _whole(parts, shape):
    return parts.transpose(0, 2, 1, 3).reshape(shape)


class Norm:
    """The forward and the gradients, and bounds on the float32 kernels' errors.

    The mean is a sum in blocks and trees, of at most 160 additions in a row for
    the sizes used here: 160 units of the mean magnitude.  The variance is taken
    around the computed mean: the same 160 units, and the square of the mean's
    error.  Half of it, and 4 roundings, are in rstd."""

    CHAIN = 160

    def __init__(self, x, groups, w, b, eps, act_name):
        self.shape, self.groups, self.act = x.shape, groups, act_name
        self.w, self.b = w, b
        p = _parts(x, groups)
        mean = p.mean((2, 3), keepdims=True)
        var = np.square(p - mean).mean((2, 3), keepdims=True)
        self.mean, self.rstd = mean[:, :, 0, 0], 1 / np.sqrt(var + eps)[:, :, 0, 0]
        rstd = 1 / np.sqrt(var + eps)
        self.mean_err = self.CHAIN * EPS * np.abs(p).mean((2, 3), keepdims=True)
        self.rstd_rel = (self.CHAIN / 2 + 6) * EPS + 0.5 * np.square(self.mean_err * rstd)
        self.xhat_parts = (p - mean) * rstd
        err = rstd * (self.mean_err + EPS * np.abs(p - mean)) + \
            np.abs(self.xhat_parts) * (self.rstd_rel + 2 * EPS)
        self.xhat, self.xhat_err = _whole(self.xhat_parts, x.shape), _whole(err, x.shape)
        self.rstd4 = rstd
        self.z = self.xhat * w + b
        self.z_err = self.xhat_err * np.abs(w) + 3 * EPS * (np.abs(self.xhat * w) + np.abs(b))

    def forward(self):
        """(y, error before the store)."""
        return act(self.z, self.act), act_tol(self.z, self.z_err, self.act)

    def gradient(self, dy):
        """dict of (gradient, error before the store)."""
        over = tuple(range(len(self.shape) - 1))
        f = slope(self.z, self.act)
        dz = dy * f
        # SiLU's slope changes by at most half for a change of z, and has its own error;
        # an element whose z lies within its error of a corner may take either slope
        f_err = 0.0
        if self.act == "silu":
            f_err = 0.5 * self.z_err + EPS * (12 + 2 * np.abs(self.z))
        elif self.act != "none":
            f_err = (np.abs(self.z) <= self.z_err) * 1.0
            if self.act == "relu6":
                f_err = np.maximum(f_err, np.abs(self.z - 6) <= self.z_err)
        dz_err = np.abs(dy) * f_err + EPS * np.abs(dz)
        n = self.CHAIN * 2
        out = {}
        t, te = np.abs(dz * self.xhat), dz_err * np.abs(self.xhat) + np.abs(dz) * self.xhat_err
        out["dw"] = (dz * self.xhat).sum(over), te.sum(over) + n * EPS * t.sum(over)
        out["db"] = dz.sum(over), dz_err.sum(over) + n * EPS * np.abs(dz).sum(over)
        g, xh = _parts(dz * self.w, self.groups), self.xhat_parts
        g_err = _parts(dz_err * np.abs(self.w) + EPS * np.abs(dz * self.w), self.groups)
        xe = _parts(self.xhat_err, self.groups)

        def mean(v):
            return v.mean((2, 3), keepdims=True)

        m1, m2 = mean(g), mean(g * xh)
        m1_err = mean(g_err) + n * EPS * mean(np.abs(g))
        m2_err = mean(g_err * np.abs(xh) + np.abs(g) * xe) + n * EPS * mean(np.abs(g * xh))
        d = g - m1 - xh * m2
        err = g_err + m1_err + np.abs(xh) * m2_err + xe * np.abs(m2) + \
            4 * EPS * (np.abs(g) + np.abs(m1) + np.abs(xh * m2))
        dx, dx_err = self.rstd4 * d, self.rstd4 * (err + (self.rstd_rel + EPS) * np.abs(d))
        out["dx"] = _whole(dx, self.shape), _whole(dx_err, self.shape)
        return out


# ------------------------------------------ matrix product in 8-bit integers
def quantize(x):
    """(numbers, scales): exact quotients of the float32 scale, halves to even."""
    most = np.abs(x).max(-1)
    with np.errstate(invalid="ignore"):
        scale = np.maximum(most.astype(np.float32) * np.float32(1 / 127), np.float32(2.0 ** -126))
        q = np.clip(np.rint(x / scale.astype(np.float64)[..., None]), -127, 127)
    bad = ~np.isfinite(most)
    q[bad], scale[bad] = 0, np.nan
    return q, scale
