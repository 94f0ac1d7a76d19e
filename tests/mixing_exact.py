"""Linear attention on numbers that lose nothing, so that a result is off by the rounding
of its store alone, whatever the order of the sums.

q, k, v and dy are whole numbers times a power of two, decays are 1 or 0 and the scale is a
power of two.  Then every product and sum is a whole number of its unit; while the sums
of the absolute values stay below 2^24 units float32 holds all of them.  Scores and states
have up to 16 bits, more than one number of a 16-bit type holds (8 or 11) and no more than two do.
"""
import numpy as np

from . import mixing_reference as ref


def whole(rng, shape, most, unit=1.0):
    """Odd and even whole numbers up to `most` in size, times `unit`."""
    return rng.integers(-most, most + 1, shape) * unit


def holds(x, bits):
    """Whether all of x are whole numbers of 2^-40 with at most `bits` bits between their
    first and their last one."""
    n = np.abs(np.asarray(x, np.float64) * 2.0 ** 40).astype(object).ravel()
    return all(int(v) == v and (v == 0 or int(v).bit_length() -
                                ((int(v) & -int(v)).bit_length() - 1) <= bits) for v in n)


def rounded(x, dtype):
    """x, which float32 holds, rounded to the type once, halves to even."""
    if dtype == "float32":
        return np.asarray(x, np.float64)
    if dtype == "float16":
        with np.errstate(over="ignore"):
            return np.asarray(x, np.float64).astype(np.float16).astype(np.float64)
    bits = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    bits = (bits + 0x7fff + (bits >> 16 & 1)) & 0xffff0000
    return bits.astype(np.uint32).view(np.float32).astype(np.float64)


def scores(q, k, scale, lo, hi):
    """[head][i][j] of a range of tokens, q (rows, H, Dk) and k (rows, KV, Dk)."""
    kh = np.repeat(k[lo:hi], q.shape[1] // k.shape[1], 1)
    return scale * np.einsum("ihd,jhd->hij", q[lo:hi], kh)


def one_number(q, k, v, h0, scale, dtype, chunk=64):
    """y of one sequence from h0 on with decays of 1, scores and states rounded to ONE number of the
    type: what the exact results have to tell from theirs."""
    group = q.shape[1] // k.shape[1]
    kh, vh = np.repeat(k, group, 1), np.repeat(v, group, 1)
    y, S = np.zeros((*q.shape[:2], v.shape[2])), h0
    for lo in range(0, len(q), chunk):
        part = slice(lo, lo + chunk)
        P = np.tril(scores(q, k, scale, lo, min(lo + chunk, len(q))))
        y[part] = np.einsum("hij,jhv->ihv", rounded(P, dtype), vh[part]) + \
            scale * np.einsum("ihd,hdv->ihv", q[part], rounded(S, dtype))
        S = S + np.einsum("jhd,jhv->hdv", kh[part], vh[part])
    return y


def majorants(q, k, v, dy, log_decay, scale, bounds, h0=None, dhT=None):
    """The sums over absolute values of the forward and of the gradients."""
    a = [np.abs(t) for t in (q, k, v)]
    h0, dhT = (None if t is None else np.abs(t) for t in (h0, dhT))
    y, hT = ref.attention(*a, log_decay, scale, bounds, h0)
    return dict(y=y, hT=hT, **ref.attention_grad(np.abs(dy), *a, log_decay, scale, bounds, h0,
                                                 dhT))


# ------------------------------------------------------ float16 with any decay
UNIT = 2.0 ** -25       # half a step of float16's smallest numbers


def _floor_of_walk(q, k, v, a, s1, bounds, back):
    """What a walk over (q, k, v) loses of numbers that are small for float16, per result
    (rows, H, Dv): the scores that a result is made of (those of a chunk's 64 tokens at
    most), each UNIT, times |v|; the elements of the state where it meets q, each UNIT, times
    s1 |q|; and what the state has lost of v, UNIT a token times |k|, which the decay reaches
    once the token's chunk has ended.  The numbers that are scaled together stay below 2^14."""
    out = np.zeros((*q.shape[:2], v.shape[2]))
    for lo, hi in bounds:
        rows = range(hi - 1, lo - 1, -1) if back else range(lo, hi)
        near_v, near_k, far = [], [], np.zeros(k.shape[1:])
        for t in rows:
            if len(near_k) == 64:
                near_v.pop(0)
                far = a[:, None] * (far + near_k.pop(0))
            else:
                far = a[:, None] * far
            near_v.append(np.abs(v[t]))
            near_k.append(np.abs(k[t]))
            lost = 1.0 + far + np.sum(near_k, 0)
            out[t] = UNIT * (np.sum(near_v, 0) +
                             s1 * np.einsum("hd,hd->h", np.abs(q[t]), lost)[:, None])
    return out


def float16_floors(r, scale):
    """dict of y, dq, dk, dv: what float16 loses of each."""
    group = r["q"].shape[1] // r["k"].shape[1]
    k, v = (np.repeat(r[n], group, 1) for n in ("k", "v"))
    q, dy, a, b = r["q"], r["dy"], ref.decay(r["log_decay"]), r["bounds"]

    def shared(x):
        return x.reshape(len(x), -1, group, x.shape[2]).sum(2)

    return dict(y=_floor_of_walk(q, k, v, a, scale, b, False),
                dq=_floor_of_walk(dy, v, k, a, scale, b, False),
                dk=shared(_floor_of_walk(v, dy, q, a, 1.0, b, True)),
                dv=shared(_floor_of_walk(k, q, dy, a, 1.0, b, True)))


def float16_tol(big, sums, tokens, floor):
    """Error of a float16 result before its store: the float32 arithmetic's, two numbers of
    22 bits for scores, states and values, and the floor."""
    return ref.attention_tol(big, sums, tokens, "float32") + 2 * 2.0 ** -22 * big + floor


def float16_bounds(r, scale):
    """{y, dq, dk, dv: (result, error before its store)}."""
    args = r["q"], r["k"], r["v"], r["log_decay"], scale, r["bounds"], r["h0"]
    want = dict(ref.attention_grad(r["dy"], *args, r["dhT"]), y=ref.attention(*args)[0])
    big = majorants(*args[:3], r["dy"], *args[3:], r["dhT"])
    assert max(np.max(big[n]) for n in ("y", "hT", "dq", "dk", "dv", "dh0")) < 2.0 ** 14
    floors, tokens = float16_floors(r, scale), max(hi - lo for lo, hi in r["bounds"])
    width = max(r["k"].shape[2], r["v"].shape[2]) + r["q"].shape[1] // r["k"].shape[1]
    return {n: (want[n], float16_tol(big[n], width, tokens, floors[n]))
            for n in ("y", "dq", "dk", "dv")}
