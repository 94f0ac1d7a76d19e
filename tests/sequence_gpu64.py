"""The sequence operators in float64 torch operations on the device, for sizes
that the walks of tests/sequence_reference.py would take too long for, and
bounds on the float32 kernels' errors.

Rows of all sequences side by side; ``Rows`` says of each row which sequence
it belongs to and where it lies in it.
"""
import torch

from .sequence_reference import EPS, ROUND, TINY


class Rows:
    def __init__(self, offsets, device="cuda"):
        offsets = torch.as_tensor(offsets, dtype=torch.int64, device=device)
        n = int(offsets[-1])
        rows = torch.arange(n, device=device)
        self.seqs, self.n = len(offsets) - 1, n
        self.start, self.end = offsets[:-1], offsets[1:]
        self.seq = torch.searchsorted(offsets[1:].contiguous(), rows, right=True)
        self.pos = rows - self.start[self.seq]
        self.left = self.end[self.seq] - 1 - rows
        self.first, self.last = (self.pos == 0)[:, None], (self.left == 0)[:, None]


def store_tol(value, err, dtype):
    """`err` before the store plus the rounding to `dtype`."""
    return err * (1 + ROUND[dtype]) + ROUND[dtype] * value.abs() + TINY[dtype] + 1e-37


def near(got, want, tol, what):
    got = got.double().reshape(want.shape)
    off = (got - want).abs()
    bad = ~(off <= tol)
    if bool(bad.any()):
        at = int(bad.flatten().nonzero()[0])
        assert False, (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}, worst error "
                       f"/ tolerance {float((off / tol).nan_to_num(float('inf')).max()):.3g}")


def act(z, name):
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0.0), "relu6": lambda: z.clamp(0.0, 6.0),
            "silu": lambda: z * torch.sigmoid(z)}[name]()


def slope(z, name):
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    return {"none": lambda: torch.ones_like(z), "relu": lambda: (z > 0).double(),
            "relu6": lambda: ((z > 0) & (z < 6)).double()}[name]()


# ------------------------------------------- causal depthwise convolution
def _row_back(x, rows, init, back):
    if back == 0:
        return x
    earlier = torch.cat([torch.zeros_like(x[:back]), x[:-back]])[:len(x)]
    outside = torch.zeros((), dtype=x.dtype, device=x.device)
    if init is not None:
        outside = init[rows.seq, (rows.pos + init.shape[1] - back).clamp(max=init.shape[1] - 1)]
    return torch.where((rows.pos >= back)[:, None], earlier, outside)


def conv(x, w, b, rows, init):
    K = w.shape[1]
    z = torch.zeros_like(x) + b
    for j in range(K):
        z += w[:, j] * _row_back(x, rows, init, K - 1 - j)
    return z


def conv_final(x, K, rows, init):
    out = torch.zeros(rows.seqs, K - 1, x.shape[1], dtype=x.dtype, device=x.device)
    for j in range(K - 1):
        at = rows.end - rows.start - (K - 1) + j
        inside = x[(rows.start + at).clamp(0, len(x) - 1)]
        before = 0.0
        if init is not None:
            before = init[torch.arange(rows.seqs, device=x.device),
                          (at + K - 1).clamp(0, K - 2)]
        out[:, j] = torch.where((at >= 0)[:, None], inside, before)
    return out


def conv_grad(dz, x, w, rows, init):
    """(dx, dw, db) for the gradient dz of the value before the activation."""
    K = w.shape[1]
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    for j in range(K):
        back = K - 1 - j
        later = torch.cat([dz[back:], torch.zeros_like(dz[:back])]) if back else dz
        dx += w[:, j] * torch.where((rows.left >= back)[:, None], later, 0.0)
        dw[:, j] = (dz * _row_back(x, rows, init, back)).sum(0)
    return dx, dw, dz.sum(0)


# ------------------------------------------------- gated linear recurrence
def _scan(a, b):
    """h[t] = a[t] h[t-1] + b[t] down the rows."""
    step = 1
    while step < len(b):
        b = torch.cat([b[:step], b[step:] + a[step:] * b[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _before(h, rows, start):
    """The row before each row, `start` (one per sequence) before the first."""
    moved = torch.cat([h[:1], h[:-1]])
    return torch.where(rows.first, start[rows.seq], moved)


class Scan:
    """The recurrence, its gradients, and bounds on the kernels' errors.

    The bounds follow the steps: a gate sigmoid(v) has a relative error of at most
    (8 + |v|) 2^-24 (the exponential's argument is rounded), and so has 1 -
    sigmoid(v); u = rate sigmoid(r) 12 more (the rate's logarithm), m = 1 - a 4
    more, and a one rounding beside m's; sqrt(1 - a^2) half of m's and 4 more.
    A step of a recurrence adds 2 roundings for the multiply-add and 3 for the
    composition of the runs.  Errors pass on through a."""

    def __init__(self, x, r, i, lam, scale, rows, h0):
        self.x, self.rows, self.scale, self.lam = x, rows, scale, lam
        C = x.shape[1]
        self.h0 = x.new_zeros(rows.seqs, C) if h0 is None else h0
        self.sr, self.si = torch.sigmoid(r), torch.sigmoid(i)
        self.cr, self.ci = torch.sigmoid(-r), torch.sigmoid(-i)     # 1 - sigmoid
        self.rate = scale * torch.nn.functional.softplus(lam, threshold=1e9)
        # softplus of a very negative lam is its exponential
        self.rate = torch.where(lam < -30, scale * torch.exp(lam), self.rate)
        log_a = -self.rate * self.sr
        self.a, self.m = torch.exp(log_a), -torch.expm1(log_a)
        self.beta = torch.sqrt(-torch.expm1(2 * log_a))
        self.e_r, self.e_i = EPS * (8 + r.abs()), EPS * (8 + i.abs())
        self.e_m = self.e_r + 16 * EPS
        self.e_a = self.e_m * self.m + EPS                  # of a, beside a itself
        self.e_beta = self.e_m / 2 + 4 * EPS
        b = self.beta * self.si * x
        e_b = (self.e_beta + self.e_i + 3 * EPS) * b.abs()
        into = torch.where(rows.first, 0.0, self.a)
        lead = self.a * self.h0[rows.seq]
        self.h = _scan(into, torch.where(rows.first, b + lead, b))
        big = _scan(into, torch.where(rows.first, b.abs() + lead.abs(), b.abs()))
        self.prev, self.prev_big = _before(self.h, rows, self.h0), _before(big, rows, self.h0.abs())
        self.err = _scan(into, (self.e_a + 5 * EPS * self.a) * self.prev_big + e_b + 2 * EPS * big)
        self.prev_err = _before(self.err, rows, torch.zeros_like(self.h0))

    def last(self):
        """(states after the sequences, bound)."""
        rows = self.rows
        if rows.n == 0:
            return self.h0, torch.zeros_like(self.h0)
        at = (rows.end - 1).clamp(min=0)
        some = (rows.end > rows.start)[:, None]
        return torch.where(some, self.h[at], self.h0), torch.where(some, self.err[at], 0.0)

    def grad(self, dy, dhT):
        """{name: (gradient, bound)} for the cotangents dy and dhT (or None)."""
        rows, a, beta, x = self.rows, self.a, self.beta, self.x
        end = torch.zeros_like(self.h0) if dhT is None else dhT
        into = torch.where(rows.last, 0.0, torch.cat([a[1:], a[:1]]))
        e_into = torch.where(rows.last, 0.0, torch.cat([self.e_a[1:], self.e_a[:1]]))

        def back(v):
            return _scan(into.flip(0), v.flip(0)).flip(0)

        g = back(torch.where(rows.last, dy + end[rows.seq], dy))
        big = back(torch.where(rows.last, dy.abs() + end[rows.seq].abs(), dy.abs()))
        after = torch.cat([big[1:], big[:1]])       # where into is not 0
        e_g = back((e_into + 5 * EPS * into) * after + 2 * EPS * big)
        out = {}
        size = beta * self.si
        out["dx"] = g * size, (e_g + (self.e_beta + self.e_i + 4 * EPS) * big) * size
        size = size * x.abs() * self.ci
        out["di"] = g * beta * x * self.si * self.ci, \
            (e_g + (self.e_beta + 2 * self.e_i + 6 * EPS) * big) * size
        held = a * self.prev
        pulled = torch.where(beta > 0, self.si * x * a * a / beta, 0.0)
        dlog = g * (held - pulled)
        held_big, pulled_big = a * self.prev_big, pulled.abs()
        dlog_big = big * (held_big + pulled_big)
        e_dlog = e_g * (held_big + pulled_big) + big * (
            a * self.prev_err + (self.e_a + 3 * EPS * a) * self.prev_big +
            (self.e_i + self.e_beta + 8 * EPS) * pulled_big +
            2 * self.e_a * (self.si * x).abs() * a / torch.where(beta > 0, beta, 1.0)) + \
            4 * EPS * dlog_big
        size = self.rate * self.sr * self.cr
        out["dr"] = -dlog * size, (e_dlog + (2 * self.e_r + 16 * EPS) * dlog_big) * size
        size = self.sr * self.scale * torch.sigmoid(self.lam)
        # the sum: 8 tokens, 16 groups of a run, then 16 rows of runs by turns
        adds = 24 + 16 + (rows.n / 128 + rows.seqs) / 16 + self.lam.abs()
        out["dlam"] = -(dlog * size).sum(0), \
            ((e_dlog + (self.e_r + (12 + adds) * EPS) * dlog_big) * size).sum(0)
        if rows.n == 0:
            out["dh0"] = end, torch.zeros_like(end)
        else:
            at, some = rows.start.clamp(max=rows.n - 1), (rows.end > rows.start)[:, None]
            p, e_p = (a * g)[at], (a * e_g + (self.e_a + 2 * EPS * a) * big)[at]
            out["dh0"] = torch.where(some, p, end), torch.where(some, e_p, 0.0)
        return out
