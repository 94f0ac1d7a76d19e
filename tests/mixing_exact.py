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
