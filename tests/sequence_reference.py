"""The sequence operators in float64 numpy, token by token, and error bounds.

Shares no code with the GPU path.  Everything is packed: x is (rows, C) and
``bounds`` the (start, end) of each sequence.  Every function also returns a
majorant, the same sums over absolute values, from which the tests take their
tolerances (unit roundoff of float32: 2^-24).
"""
import numpy as np

EPS = 2.0 ** -24
ROUND = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float32": 0.0, "float16": 2.0 ** -25, "bfloat16": 0.0}   # subnormal spacing / 2


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def softplus(v):
    return np.logaddexp(0.0, v)


def act(z, name):
    return {"none": lambda: z, "relu": lambda: np.maximum(z, 0.0),
            "relu6": lambda: np.clip(z, 0.0, 6.0), "silu": lambda: z * sigmoid(z)}[name]()


def slope(z, name):
    if name == "silu":
        s = sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    return {"none": np.ones_like(z), "relu": (z > 0) * 1.0,
            "relu6": ((z > 0) & (z < 6)) * 1.0}[name]


def bounds_of(offsets):
    return list(zip(offsets[:-1], offsets[1:]))


# ------------------------------------------- causal depthwise convolution
def conv(x, w, b, bounds, init):
    """(z, majorant of z, final rows); init (S, K-1, C) or None."""
    C, K = w.shape
    z, big = np.zeros_like(x), np.zeros_like(x)
    final = np.zeros((len(bounds), K - 1, C))
    for s, (lo, hi) in enumerate(bounds):
        carried = np.zeros((K - 1, C)) if init is None else init[s]
        line = np.concatenate([carried, x[lo:hi]])
        for t in range(hi - lo):
            terms = line[t:t + K] * w.T
            z[lo + t] = terms.sum(0) + b
            big[lo + t] = np.abs(terms).sum(0) + np.abs(b)
        final[s] = line[len(line) - (K - 1):]
    return z, big, final


def conv_grad(dy, x, w, b, bounds, init, dfinal, act_name):
    """dict of (gradient, majorant)."""
    C, K = w.shape
    z, _, _ = conv(x, w, b, bounds, init)
    out = {n: [np.zeros(s), np.zeros(s)] for n, s in
           (("dx", x.shape), ("dw", w.shape), ("db", (C,)),
            ("dinit", (len(bounds), K - 1, C)))}
    for s, (lo, hi) in enumerate(bounds):
        carried = np.zeros((K - 1, C)) if init is None else init[s]
        line = np.concatenate([carried, x[lo:hi]])
        for kind in (0, 1):
            f = np.abs if kind else (lambda v: v)
            dline = np.zeros_like(line)
            for t in range(hi - lo):
                dz = f(dy[lo + t] * slope(z[lo + t], act_name))
                dline[t:t + K] += f(w.T) * dz
                out["dw"][kind] += (f(line[t:t + K]) * dz).T
                out["db"][kind] += dz
            if dfinal is not None:
                dline[len(line) - (K - 1):] += f(dfinal[s])
            out["dinit"][kind][s] = dline[:K - 1]
            out["dx"][kind][lo:hi] = dline[K - 1:]
    return out


# ------------------------------------------------- gated linear recurrence
def gates(x, r, i, lam, scale):
    log_a = -scale * softplus(lam) * sigmoid(r)
    a = np.exp(log_a)
    beta = np.sqrt(-np.expm1(2 * log_a))
    return a, beta, sigmoid(i)


def scan(x, r, i, lam, scale, bounds, h0):
    """(h, bound on the float32 error of h, final states, its bound).

    One step in float32: a has a relative error of at most (4 + 32 m) 2^-24,
    m = 1 - a (a is 1 - m rounded once, m = u (1 - u/2 ...) good to 32 2^-24 with
    the gate's sigmoid and the logits of |r| <= 16 used here), beta sigma(i) x
    of 48 2^-24 at most, and the fused multiply-add of one rounding.  Errors
    pass on through a."""
    a, beta, si = gates(x, r, i, lam, scale)
    b = beta * si * x
    h, err = np.zeros_like(x), np.zeros_like(x)
    C = x.shape[1]
    last, last_err = np.zeros((len(bounds), C)), np.zeros((len(bounds), C))
    for s, (lo, hi) in enumerate(bounds):
        cur = np.zeros(C) if h0 is None else h0[s].copy()
        big, e = np.abs(cur), np.zeros(C)
        for t in range(lo, hi):
            e = a[t] * e + EPS * ((6 + 32 * (1 - a[t])) * a[t] * big + 48 * np.abs(b[t]))
            big = a[t] * big + np.abs(b[t])
            cur = a[t] * cur + b[t]
            h[t], err[t] = cur, e
        last[s], last_err[s] = cur, e
    return h, err, last, last_err


def scan_grad(dy, x, r, i, lam, scale, bounds, h0, dhT):
    """dict of (gradient, majorant)."""
    a, beta, si = gates(x, r, i, lam, scale)
    sr, k = sigmoid(r), scale * softplus(lam)
    C = x.shape[1]
    out = {n: [np.zeros_like(x), np.zeros_like(x)] for n in ("dx", "dr", "di")}
    out["dlam"] = [np.zeros(C), np.zeros(C)]
    out["dh0"] = [np.zeros((len(bounds), C)), np.zeros((len(bounds), C))]
    for kind in (0, 1):
        f = np.abs if kind else (lambda v: v)
        for s, (lo, hi) in enumerate(bounds):
            start = np.zeros(C) if h0 is None else f(h0[s])
            hs, cur = [], start
            for t in range(lo, hi):
                hs.append(cur)
                cur = a[t] * cur + f(beta[t] * si[t] * x[t])
            p = np.zeros(C) if dhT is None else f(dhT[s])
            for t in range(hi - 1, lo - 1, -1):
                g = f(dy[t]) + p
                with np.errstate(divide="ignore", invalid="ignore"):
                    back = np.where(beta[t] > 0, f(si[t] * x[t]) * a[t] ** 2 / beta[t], 0.0)
                dlog = g * (a[t] * hs[t - lo] + back) if kind else \
                    g * (a[t] * hs[t - lo] - back)
                out["dx"][kind][t] = g * beta[t] * si[t]
                out["di"][kind][t] = g * beta[t] * f(x[t]) * si[t] * (1 - si[t])
                out["dr"][kind][t] = f(-dlog * k * sr[t] * (1 - sr[t]))
                out["dlam"][kind] += f(-dlog * sr[t] * scale * sigmoid(lam))
                p = a[t] * g
            out["dh0"][kind][s] = p
    return out


# --------------------------------- matrix product with bias, activation, residual
def linear(x, w, b):
    """(z, majorant)."""
    z, big = x @ w.T, np.abs(x) @ np.abs(w).T
    if b is not None:
        z, big = z + b, big + np.abs(b)
    return z, big


def linear_grad(dy, x, w, z, act_name):
    dz = dy if act_name == "none" else dy * slope(z, act_name)
    return {"dz": dz, "dx": (dz @ w, np.abs(dz) @ np.abs(w)),
            "dw": (dz.T @ x, np.abs(dz).T @ np.abs(x)), "db": (dz.sum(0), np.abs(dz).sum(0))}


# ------------------------------------------------------------- tolerances
def act_tol(z, z_err, name):
    """Error of act(z) in float32 for an error z_err of z: the activations'
    slopes are below 1.1; SiLU adds the relative error of its exponential
    (|z| 2^-23 from the argument), reciprocal and products: (8 + 2|z|) 2^-24."""
    tol = 1.1 * z_err
    if name == "silu":
        tol = tol + EPS * (8 + 2 * np.abs(z)) * np.abs(act(z, "silu"))
    return tol


def store_tol(value, err, dtype):
    """`err` before the store plus the rounding to `dtype`."""
    return err * (1 + ROUND[dtype]) + ROUND[dtype] * np.abs(value) + TINY[dtype] + 1e-37
