"""GPU parity of the mixing operators (linear attention, group normalisation,
8-bit products) against float64 references.

Tolerances come from the number of roundings on the way to each result
(tests/mixing_reference.py), never from what a run gave.  Inputs are drawn in
float64 and rounded to the tensors' type first.
"""
import numpy as np
import pytest

import depthwise_convolution_amd as dw

from . import mixing_reference as ref
from .sequence_reference import bounds_of

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "float16", "bfloat16"]
# sequences of a packed batch: of no token, of one, around a chunk, and longer
RAGGED = [0, 1, 0, 2, 31, 33, 63, 64, 65, 1, 300, 0]


@pytest.fixture(scope="module")
def torch():
    import torch as t
    if not t.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    return t


def _gpu(torch, a, dtype="float32"):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", getattr(torch, dtype))


def _back(t):
    return t.detach().double().cpu().numpy()


def _draw(torch, rng, shape, dtype, scale=1.0):
    """(GPU tensor, its values in float64)."""
    t = _gpu(torch, rng.standard_normal(shape) * scale, dtype)
    return t, _back(t)


def _near(got, want, tol, what):
    got = _back(got).reshape(want.shape)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst error / tolerance "
                           f"{np.nanmax(np.abs(got - want) / tol):.3g}, first at "
                           f"{np.argwhere(bad)[0].tolist()}")


def _offsets(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)


def _wide(torch, t, pad=5):
    """The same values as a column range of a wider tensor, NaN beside it."""
    rows, width = t.shape[:-2], t.shape[-2] * t.shape[-1]
    big = torch.full((*rows, width + 2 * pad), float("nan"), dtype=t.dtype, device=t.device)
    view = big[..., pad:pad + width].unflatten(-1, t.shape[-2:])
    view.copy_(t)
    return view


# ---------------------------- linear attention with a decay for each head
ATTENTION_CASES = [
    # (lengths or (S, T), H, KV, Dk, Dv, carry, strided)
    (RAGGED, 4, 2, 24, 17, True, True),
    (RAGGED, 2, 2, 64, 64, False, False),
    ((2, 150), 2, 2, 16, 16, False, False),
    ((1, 1), 3, 3, 1, 1, True, False),
    ((5, 1), 2, 1, 64, 128, True, True),
    ((1, 700), 1, 1, 64, 64, True, False),                  # cut into segments
    ([70, 600, 0, 5, 530], 2, 1, 128, 128, True, False),    # and packed ones
    ([1100], 1, 1, 96, 80, False, True),
    ((2, 65), 2, 1, 130, 65, True, False),
    ((1, 300), 1, 1, 256, 256, False, False),
    ((2, 129), 6, 2, 40, 72, True, False),
    ((3, 64), 3, 1, 128, 64, False, True),
    ((1, 33), 2, 2, 3, 200, True, False),
    ((2, 0), 2, 2, 16, 16, True, False),
    ([0, 0, 0], 2, 1, 16, 16, True, False),
]


def _attention_inputs(torch, case, dtype, seed):
    layout, H, KV, Dk, Dv, carry, strided = case
    rng = np.random.default_rng(seed)
    packed = isinstance(layout, list)
    offsets = _offsets(layout) if packed else _offsets([layout[1]] * layout[0])
    lead = (int(offsets[-1]),) if packed else layout
    S = len(offsets) - 1
    # from no memory to all: at most 0, above it, and minus infinity among them
    logs = np.array([-0.02, 0.0, -1.0, 0.5, -np.inf, -8.0])
    g, r = {}, {}
    for name, shape in (("q", (H, Dk)), ("k", (KV, Dk)), ("v", (KV, Dv)), ("dy", (H, Dv))):
        g[name], r[name] = _draw(torch, rng, (*lead, *shape), dtype)
        r[name] = r[name].reshape(-1, *shape)
        if strided:
            g[name] = _wide(torch, g[name])
    g["log_decay"] = _gpu(torch, np.resize(np.roll(logs, seed), H))
    r["log_decay"] = _back(g["log_decay"])
    for name in ("h0", "dhT"):
        g[name], r[name] = _draw(torch, rng, (S, H, Dk, Dv), "float32") if carry else (None, None)
    g["off"] = _gpu(torch, offsets, "int32") if packed else None
    r["bounds"] = bounds_of(offsets)
    return g, r


def _abs(r, *names):
    return [None if r[n] is None else np.abs(r[n]) for n in names]


def _longest(r):
    return max(hi - lo for lo, hi in r["bounds"])


def _floor16(dtype, big_scores, v, big_state, q):
    """What float16 loses of scores and state elements far below the largest of those
    that are scaled together: 2^-23 of it, times what it is multiplied by."""
    if dtype != "float16" or not len(v):
        return 0.0
    return 2.0 ** -23 * (big_scores * 64 * np.abs(v).max() + big_state * np.abs(q).max() * 256)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(ATTENTION_CASES)))
def test_attention(torch, case, dtype):
    spec = ATTENTION_CASES[case]
    Dk, scale = spec[3], 0.7 * spec[3] ** -0.5
    print(f"\n[case] linear_attention {spec} {dtype}", flush=True)
    g, r = _attention_inputs(torch, spec, dtype, case)
    y, hT = dw.linear_attention(g["q"], g["k"], g["v"], g["log_decay"], h0=g["h0"],
                                offsets=g["off"], scale=scale)
    torch.cuda.synchronize()
    want, state = ref.attention(r["q"], r["k"], r["v"], r["log_decay"], scale, r["bounds"],
                                r["h0"])
    qa, ka, va, ha = _abs(r, "q", "k", "v", "h0")
    big, big_state = ref.attention(qa, ka, va, r["log_decay"], scale, r["bounds"], ha)
    tokens = _longest(r)
    floor = _floor16(dtype, scale * 64 * Dk, va, scale * np.max(big_state, initial=0.0), qa)
    tol = ref.attention_tol(big, Dk, tokens, dtype, floor)
    _near(y, want, ref.store_tol(want, tol, dtype), "y")
    small = 2.0 ** -22 * 64 * 25 if dtype == "float16" else 0.0
    _near(hT, state, ref.store_tol(state, ref.attention_tol(big_state, 0, tokens, dtype, small,
                                                            True), "float32"), "hT")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(ATTENTION_CASES)))
def test_attention_grad(torch, case, dtype):
    spec = ATTENTION_CASES[case]
    _, H, KV, Dk, Dv, carry, _ = spec
    scale = 0.7 * Dk ** -0.5
    print(f"\n[case] linear_attention_grad {spec} {dtype}", flush=True)
    g, r = _attention_inputs(torch, spec, dtype, case)
    got = dw.linear_attention_grad(g["dy"], g["q"], g["k"], g["v"], g["log_decay"], h0=g["h0"],
                                   dhT=g["dhT"], offsets=g["off"], scale=scale)
    torch.cuda.synchronize()
    want = ref.attention_grad(r["dy"], r["q"], r["k"], r["v"], r["log_decay"], scale,
                              r["bounds"], r["h0"], r["dhT"])
    big = ref.attention_grad(*_abs(r, "dy", "q", "k", "v"), r["log_decay"], scale, r["bounds"],
                             *_abs(r, "h0", "dhT"))
    tokens = _longest(r)
    width = max(Dk, Dv)
    top = max((np.max(b, initial=0.0) for b in big.values()), default=0.0)
    floor = _floor16(dtype, 64.0 * width, r["v"], 4 * top, r["q"])
    for name, t in zip(("dq", "dk", "dv"), got):
        # heads that share a key: each of their sums has its own error, and one more
        tol = ref.attention_tol(big[name], width + H // KV, tokens, dtype, floor)
        _near(t, want[name], ref.store_tol(want[name], tol, dtype), name)
    assert (got[3] is None) == (not carry)
    if carry:
        small = 2.0 ** -22 * 64 * 25 if dtype == "float16" else 0.0
        tol = ref.attention_tol(big["dh0"], 0, tokens, dtype, small, True)
        _near(got[3], want["dh0"], ref.store_tol(want["dh0"], tol, "float32"), "dh0")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seqs,H,KV,Dk,Dv", [(1, 1, 1, 1, 1), (3, 4, 2, 24, 17), (2, 2, 2, 256, 256),
                                             (5, 6, 1, 64, 128), (2, 3, 3, 128, 4)])
def test_attention_step(torch, seqs, H, KV, Dk, Dv, dtype):
    g, r = _attention_inputs(torch, ((seqs, 1), H, KV, Dk, Dv, True, True), dtype, Dk)
    h = g["h0"].clone()
    y = dw.linear_attention_step(g["q"][:, 0], g["k"][:, 0], g["v"][:, 0], g["log_decay"], h)
    torch.cuda.synchronize()
    scale = Dk ** -0.5
    want, state = ref.attention(r["q"], r["k"], r["v"], r["log_decay"], scale, r["bounds"],
                                r["h0"])
    big, big_state = ref.attention(*_abs(r, "q", "k", "v"), r["log_decay"], scale, r["bounds"],
                                   np.abs(r["h0"]))
    # the decay (2 and 1.25 of its exponent, at most 8 here or nothing), a product, a sum
    _near(h, state, 16 * ref.EPS * big_state, "h")
    _near(y, want, ref.store_tol(want, (2 * Dk + 20) * ref.EPS * big, dtype), "y")


def test_attention_defaults_and_the_prompt_in_parts(torch):
    """scale is Dk ** -0.5; a prompt taken in three parts and then token by token gives
    what it gives at once, to the tolerances of both."""
    rng = np.random.default_rng(8)
    for dtype in DTYPES:
        shape = (2, 205, 3, 48)
        (q, qr), (k, kr), (v, vr) = (_draw(torch, rng, shape, dtype) for _ in range(3))
        g = torch.tensor([-0.01, -0.3, 0.0], device="cuda")
        whole, last = dw.linear_attention(q, k, v, g)
        same, _ = dw.linear_attention(q, k, v, g, scale=48 ** -0.5)
        assert torch.equal(whole, same)
        parts, h = [], None
        for lo, hi in ((0, 64), (64, 65), (65, 200)):
            y, h = dw.linear_attention(q[:, lo:hi].contiguous(), k[:, lo:hi].contiguous(),
                                       v[:, lo:hi].contiguous(), g, h0=h)
            parts.append(y)
        for t in range(200, 205):
            parts.append(dw.linear_attention_step(q[:, t].contiguous(), k[:, t].contiguous(),
                                                  v[:, t].contiguous(), g, h)[:, None])
        both = torch.cat(parts, 1)
        flat = [np.abs(t).reshape(-1, 3, 48) for t in (qr, kr, vr)]
        big, bs = ref.attention(*flat, _back(g), 48 ** -0.5, [(0, 205), (205, 410)], None)
        tol = ref.store_tol(big, ref.attention_tol(big, 48, 205, dtype, 2.0 ** -20 * big.max()),
                            dtype)
        _near(both, _back(whole).reshape(big.shape), 2 * tol, "parts")
        _near(h, _back(last), 2 * ref.attention_tol(bs, 0, 205, dtype, 2.0 ** -22 * 1600, True),
              "state")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [24, 64, 128])
def test_attention_keeps_infinities_from_earlier_tokens(torch, dtype, D):
    """An infinity or NaN of token 77 leaves the tokens before it, the other heads and
    the other sequences as they were, bit for bit; a token's infinite value reaches
    the columns that it is in."""
    rng = np.random.default_rng(3)
    q, k, v = (_draw(torch, rng, (2, 200, 2, D), dtype)[0] for _ in range(3))
    g = torch.tensor([-0.01, -0.5], device="cuda")
    y0, h0 = dw.linear_attention(q, k, v, g)
    grads0 = dw.linear_attention_grad(y0, q, k, v, g)
    for name in ("q", "k", "v"):
        for bad in (float("inf"), float("nan")):
            t = dict(q=q.clone(), k=k.clone(), v=v.clone())
            t[name][0, 77, 1, 5] = bad
            y, h = dw.linear_attention(t["q"], t["k"], t["v"], g)
            assert torch.equal(y[1], y0[1]) and torch.equal(h[1], h0[1])
            assert torch.equal(y[0, :, 0], y0[0, :, 0])
            assert torch.equal(y[0, :77], y0[0, :77])
            assert not torch.isfinite(y[0, 77, 1]).all()
            if name == "q":
                assert torch.equal(y[0, 78:], y0[0, 78:]) and torch.equal(h, h0)
            if name == "v":
                rest = [c for c in range(D) if c != 5]
                assert torch.equal(y[0, :, 1][:, rest], y0[0, :, 1][:, rest])
                assert not torch.isfinite(y[0, 77:, 1, 5]).any()
                # one infinite term among finite ones has the sign of its score
                score = (q[0, 77, 1].double() * k[0, 77, 1].double()).sum()
                if bad == float("inf"):
                    assert y[0, 77, 1, 5] == (bad if score > 0 else -bad)
            dq, dk, dv, _ = dw.linear_attention_grad(y0, t["q"], t["k"], t["v"], g)
            # what a token brings reaches the gradients of keys before it only
            if name == "q":
                assert torch.equal(dk[0, 78:], grads0[1][0, 78:])
                assert torch.equal(dv[0, 78:], grads0[2][0, 78:])
            else:
                assert torch.equal(dq[0, :77], grads0[0][0, :77])


def test_attention_float16_range(torch):
    """float16 scores and states beyond its largest number, and far below its smallest
    normal one, keep the precision of the rest."""
    rng = np.random.default_rng(4)
    g = torch.tensor([-0.01, 0.0], device="cuda")
    for grow in (2.0 ** -12, 1.0, 2.0 ** 7):
        q, k = (_draw(torch, rng, (1, 300, 2, 64), "float16", grow) for _ in range(2))
        v = _draw(torch, rng, (1, 300, 2, 64), "float16", min(1.0, 2.0 ** -8 / grow))
        scale = 0.125 * min(1.0 / grow, 2.0 ** 20)
        y, h = dw.linear_attention(q[0], k[0], v[0], g, scale=scale)
        args = [t[1].reshape(-1, 2, 64) for t in (q, k, v)]
        want, state = ref.attention(*args, _back(g), scale, [(0, 300)], None)
        big, bs = ref.attention(*map(np.abs, args), _back(g), scale, [(0, 300)], None)
        floor = 2.0 ** -23 * (scale * np.abs(args[0]).max() * np.abs(args[1]).max() * 64 * 64 *
                              np.abs(args[2]).max() + scale * bs.max() *
                              np.abs(args[0]).max() * 64)
        tol = ref.attention_tol(big, 64, 300, "float16", floor)
        _near(y, want, ref.store_tol(want, tol, "float16"), f"y at {grow}")
        small = 2.0 ** -22 * 64 * np.abs(args[1]).max() * np.abs(args[2]).max()
        _near(h, state, ref.attention_tol(bs, 0, 300, "float16", small, True), f"h at {grow}")


def test_attention_writes_its_own_columns(torch):
    """Results into column ranges of one tensor, and gradients: nothing else written,
    and arrays that are not wanted may be left out."""
    rng = np.random.default_rng(5)
    for dtype in DTYPES:
        q, k, v = (_draw(torch, rng, (70, 2, 24), dtype)[0] for _ in range(3))
        off = torch.tensor([0, 30, 70], dtype=torch.int32, device="cuda")
        g = torch.tensor([-0.1, -0.2], device="cuda")
        y, _ = dw.linear_attention(q, k, v, g, offsets=off)
        out = torch.full((70, 60), 7.0, dtype=q.dtype, device="cuda")
        dw.dwconv_attention_fwd(q, k, v, g, out[:, 6:54].unflatten(-1, (2, 24)), offsets=off)
        assert torch.equal(out[:, 6:54], y.flatten(1))
        assert (out[:, :6] == 7).all() and (out[:, 54:] == 7).all()
        dq, dk, dv, _ = dw.linear_attention_grad(y, q, k, v, g, offsets=off)
        n = dw.dwconv_attention_workspace_size(True, q.dtype, 2, 70, True, 2, 2, 24, 24)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        both = torch.full((70, 3, 2, 24), 7.0, dtype=q.dtype, device="cuda")
        dw.dwconv_attention_grad(y, q, k, v, g, None, both[:, 1], None, workspace=ws, offsets=off)
        assert torch.equal(both[:, 1], dk) and (both[:, 0] == 7).all() and (both[:, 2] == 7).all()
        dw.dwconv_attention_grad(y, q, k, v, g, both[:, 0], None, both[:, 2], workspace=ws,
                                 offsets=off)
        assert torch.equal(both, torch.stack([dq, dk, dv], 1))


# ------------------------------------- group normalisation with an activation
NORM_CASES = [
    # (shape, groups, act)
    ((5, 7, 9, 24), 4, "silu"), ((2, 33, 31, 320), 32, "silu"), ((1, 60, 50, 256), 32, "none"),
    ((300, 2048), 16, "silu"), ((33, 96), 8, "none"), ((33, 2048), 1, "relu"),
    ((7, 5120), 1, "none"), ((3, 40000), 2, "relu6"), ((200, 33), 3, "silu"),
    ((9, 3, 5001), 3, "silu"), ((4, 2, 4096), 1, "silu"), ((70, 2, 16), 2, "none"),
    ((2, 300, 30), 30, "silu"), ((1, 5, 16), 1, "relu"), ((3, 1, 1, 48), 12, "none"),
    ((500, 1600), 20, "silu"), ((1, 4000, 8), 2, "silu"), ((8, 400, 12), 4, "none"),
    ((600, 3, 4), 1, "silu"), ((2, 2500), 2500 // 500, "silu"),
]


def _norm_inputs(torch, case, dtype, seed):
    shape, groups, act = case
    rng = np.random.default_rng(seed)
    C = shape[-1]
    x, _ = _draw(torch, rng, shape, "float64")
    x = (x * 1.5 + _gpu(torch, rng.standard_normal(C) * 3, "float64")).to(getattr(torch, dtype))
    w, wr = _draw(torch, rng, (C,), "float32")
    b, br = _draw(torch, rng, (C,), "float32")
    dy, dyr = _draw(torch, rng, shape, dtype)
    return x, w + 1, b, dy, ref.Norm(_back(x), groups, wr * 0 + _back(w + 1), br, 1e-5, act), dyr


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(NORM_CASES)))
def test_group_norm(torch, case, dtype):
    shape, groups, act = spec = NORM_CASES[case]
    print(f"\n[case] group_norm {spec} {dtype}", flush=True)
    x, w, b, dy, r, dyr = _norm_inputs(torch, spec, dtype, case)
    y, stats = dw.group_norm(x, groups, w, b, act=act, save_stats=True)
    grads = dw.group_norm_grad(dy, x, stats, groups, w, b, act=act)
    torch.cuda.synchronize()
    want, tol = r.forward()
    _near(y, want, ref.store_tol(want, tol, dtype), "y")
    _near(stats[..., 0], r.mean, r.mean_err[:, :, 0, 0] + 1e-37, "mean")
    _near(stats[..., 1], r.rstd, r.rstd * r.rstd_rel[:, :, 0, 0], "rstd")
    want = r.gradient(dyr)
    for name, t, kind in zip(("dx", "dw", "db"), grads, (dtype, "float32", "float32")):
        _near(t, want[name][0], ref.store_tol(want[name][0], want[name][1], kind), name)
    assert torch.equal(y, dw.group_norm(x, groups, w, b, act=act))


def test_group_norm_without_scale_in_place_and_in_column_ranges(torch):
    rng = np.random.default_rng(2)
    for shape in ((40, 96), (3, 50, 96)):
        for dtype in DTYPES:
            x, xr = _draw(torch, rng, shape, dtype)
            one, zero = torch.ones(96, device="cuda"), torch.zeros(96, device="cuda")
            y, stats = dw.group_norm(x, 8, one, zero, act="silu", save_stats=True)
            assert torch.equal(y, dw.group_norm(x, 8, act="silu"))
            dy = _draw(torch, rng, shape, dtype)[0]
            a = dw.group_norm_grad(dy, x, stats, 8, one, zero, act="silu")
            b = dw.group_norm_grad(dy, x, stats, 8, act="silu")
            assert all(torch.equal(s, t) for s, t in zip(a, b))
            P = shape[1] if len(shape) == 3 else 1
            n = dw.dwconv_norm_workspace_size(False, x.dtype, shape[0], P, 96, 8)
            ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
            big = torch.full((*shape[:-1], 110), 7.0, dtype=x.dtype, device="cuda")
            view = big[..., 6:102]
            view.copy_(x)
            dw.dwconv_norm_fwd(view, 8, None, None, view, act="silu", workspace=ws)
            assert torch.equal(view, y) and (big[..., :6] == 7).all() and \
                (big[..., 102:] == 7).all()
            n = dw.dwconv_norm_workspace_size(True, x.dtype, shape[0], P, 96, 8)
            ws = torch.empty(n, dtype=torch.uint8, device="cuda")
            d = dy.clone()
            dw.dwconv_norm_grad(d, x, stats, 8, None, None, d, None, None, act="silu",
                                workspace=ws)
            assert torch.equal(d, a[0])
            db = torch.empty(96, device="cuda")
            dw.dwconv_norm_grad(dy, x, stats, 8, None, None, None, None, db, act="silu",
                                workspace=ws)
            assert torch.equal(db, a[2])


def test_group_norm_of_nothing_and_of_strange_values(torch):
    x = torch.empty(0, 16, device="cuda")
    y, stats = dw.group_norm(x, 4, save_stats=True)
    dx, dw_, db = dw.group_norm_grad(x, x, stats, 4)
    assert y.shape == (0, 16) and stats.shape == (0, 4, 2) and dx.shape == (0, 16)
    assert (dw_ == 0).all() and (db == 0).all()
    for dtype in DTYPES:
        for shape in ((6, 32), (6, 40, 32)):
            x = torch.ones(shape, dtype=getattr(torch, dtype), device="cuda")
            assert (dw.group_norm(x, 4) == 0).all()         # no spread: xhat is 0
            x[2, ..., 9] = float("nan")
            x[3, ..., 0] = float("inf")
            y = dw.group_norm(x, 4)
            odd = ~torch.isfinite(y.reshape(6, -1, 4, 8)).all(1).all(-1)
            assert odd[2].tolist() == [False, True, False, False]
            assert odd[3].tolist() == [True, False, False, False]
            assert not odd[[0, 1, 4, 5]].any()
    # a mean far from 0: the variance is not a difference of large numbers
    rng = np.random.default_rng(0)
    for shape in ((20, 256), (2, 900, 16)):
        x, xr = _draw(torch, rng, shape, "float32")
        x = x + 1000.0
        r = ref.Norm(_back(x), 2, np.ones(shape[-1]), np.zeros(shape[-1]), 1e-5, "none")
        want, tol = r.forward()
        _near(dw.group_norm(x, 2), want, ref.store_tol(want, tol, "float32"), "far mean")


def test_group_norm_many_instances(torch):
    """More instances than are summed at once for dw and db."""
    rng = np.random.default_rng(6)
    for shape, groups in (((1500, 3, 8), 2), ((9000, 8), 1)):
        x, xr = _draw(torch, rng, shape, "float32")
        dy, dyr = _draw(torch, rng, shape, "float32")
        r = ref.Norm(xr, groups, np.ones(8), np.zeros(8), 1e-5, "silu")
        y, stats = dw.group_norm(x, groups, act="silu", save_stats=True)
        got = dw.group_norm_grad(dy, x, stats, groups, act="silu")
        want = r.gradient(dyr)
        for name, t in zip(("dx", "dw", "db"), got):
            _near(t, want[name][0], ref.store_tol(*want[name], "float32"), name)


# ------------------------------------------ matrix product in 8-bit integers
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,scale", [(5, 7, 1.0), (3, 2048, 1e-3), (1100, 600, 1.0),
                                       (1030, 5000, 3.0), (2, 130001, 1.0), (1500, 33, 1e-4)])
def test_quantize_rows(torch, M, K, scale, dtype):
    rng = np.random.default_rng(K)
    x, xr = _draw(torch, rng, (M, K), dtype, scale)
    x[0], xr[0] = 0, 0
    q, s = dw.quantize_rows(x)
    want, scales = ref.quantize(xr)
    assert np.array_equal(s.cpu().numpy(), scales)
    assert np.array_equal(q.cpu().numpy(), want)


def test_quantize_rows_at_halves_and_at_the_ends(torch):
    row = [127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, 126.49999, 1e-30, -127.0]
    x = torch.tensor([row, [v * 2.0 ** -100 for v in row], [v * 2.0 ** 100 for v in row],
                      [v * 2.0 ** -140 for v in row], [0.0] * 10, [float("nan")] + row[1:],
                      row[:9] + [float("-inf")]], device="cuda")
    q, s = dw.quantize_rows(x)
    want, scales = ref.quantize(_back(x))
    assert np.array_equal(q.cpu().numpy(), want)
    assert np.array_equal(s.cpu().numpy(), scales, equal_nan=True)
    # into rows of a wider tensor, from a column range
    wide = torch.full((7, 16), 99, dtype=torch.int8, device="cuda")
    dw.dwconv_quantize_rows(x[:, 1:8], wide[:, 4:11], s)
    want, scales = ref.quantize(_back(x[:, 1:8]))
    assert np.array_equal(wide[:, 4:11].cpu().numpy(), want)
    assert (wide[:, :4] == 99).all() and (wide[:, 11:] == 99).all()


I8_CASES = [
    # (M, N, K, act, bias, res)
    (1, 50, 33, "none", True, False), (8, 256, 512, "silu", True, True),
    (16, 100, 2048, "relu", False, True), (40, 100, 512, "silu", True, False),
    (64, 77, 1000, "relu6", True, True), (130, 200, 300, "none", False, False),
    (300, 256, 1024, "silu", True, True), (513, 400, 208, "relu6", True, False),
    (1000, 520, 272, "none", True, True), (100, 64, 16384, "silu", False, False),
    (257, 513, 130, "silu", True, True), (0, 8, 16, "none", True, False), (3, 1, 1, "none", True, True),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(I8_CASES)))
def test_linear_i8(torch, case, dtype):
    M, N, K, act, bias, res = spec = I8_CASES[case]
    print(f"\n[case] linear_i8 {spec} {dtype}", flush=True)
    rng = np.random.default_rng(case)
    x, xr = _draw(torch, rng, (M, K), dtype)
    w, _ = _draw(torch, rng, (N, K), "float32", K ** -0.5)
    wq, ws = dw.quantize_rows(w)
    b, br = _draw(torch, rng, (N,), "float32") if bias else (None, 0.0)
    rs, rr = _draw(torch, rng, (M, N), dtype) if res else (None, 0.0)
    y = dw.linear_i8(x, wq, ws, b, act=act, res=rs)
    torch.cuda.synchronize()
    if M == 0:
        assert y.shape == (0, N)
        return
    q, s = ref.quantize(xr)
    z0 = (q @ _back(wq).T) * s.astype(np.float64)[:, None] * _back(ws)
    z = z0 + br
    # the integers are exact; their sum, the factors' product and theirs are rounded
    z_err = 4 * ref.EPS * np.abs(z0) + ref.EPS * np.abs(z)
    want, tol = ref.act(z, act) + rr, ref.act_tol(z, z_err, act)
    tol = tol + ref.EPS * np.abs(want)
    _near(y, want, ref.store_tol(want, tol, dtype), "y")
    # the same from numbers made beforehand, and from rows of a wider tensor
    xq, xs = dw.quantize_rows(x)
    assert torch.equal(y, dw.linear_i8(xq, wq, ws, b, act=act, res=rs, x_scale=xs, dtype=x.dtype))
    wide = torch.full((M, K + 9), 55, dtype=torch.int8, device="cuda")
    wide[:, 3:K + 3] = xq
    far = torch.full((N, K + 5), -77, dtype=torch.int8, device="cuda")
    far[:, 1:K + 1] = wq
    assert torch.equal(y, dw.linear_i8(wide[:, 3:K + 3], far[:, 1:K + 1], ws, b, act=act, res=rs,
                                       x_scale=xs, dtype=x.dtype))


def test_linear_i8_extremes(torch):
    """The largest sums that 32 bits hold; rows that are not finite stay by themselves."""
    K = dw.I8_MAX_K
    x = torch.full((2, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(3, device="cuda")
    y = dw.linear_i8(x, w, one, x_scale=one[:2], dtype=torch.float32)
    assert (y.double() == np.float32(128 * 128 * K)).all()
    for M in (4, 200):
        x = torch.ones(M, 64, device="cuda")
        x[1, 3], x[2, 60] = float("inf"), float("nan")
        wq, ws = dw.quantize_rows(torch.full((72, 64), 0.5, device="cuda"))
        y = dw.linear_i8(x, wq, ws)
        assert torch.isnan(y[1:3]).all() and torch.isfinite(y[[0, 3]]).all()


# ------------------------------------------------------------ all of them
def _everything(torch, dtype, seed=0):
    """(inputs that a caller may change, call) of every operator, as in a block."""
    rng = np.random.default_rng(seed)
    q, k, v = (_draw(torch, rng, (1000, 2, 64), dtype)[0] for _ in range(3))
    off = torch.tensor([0, 700, 700, 1000], dtype=torch.int32, device="cuda")
    g = torch.tensor([-0.01, -0.3], device="cuda")
    img, dimg = (_draw(torch, rng, (2, 300, 48), dtype)[0] for _ in range(2))
    tok, dtok = (_draw(torch, rng, (100, 96), dtype)[0] for _ in range(2))
    w = torch.ones(48, device="cuda")
    few, many = _draw(torch, rng, (8, 128), dtype)[0], _draw(torch, rng, (300, 128), dtype)[0]
    wq, ws = dw.quantize_rows(_draw(torch, rng, (96, 128), "float32")[0])
    h = torch.zeros(1000, 2, 64, 64, device="cuda")[:5].contiguous()

    def call():
        y, hT = dw.linear_attention(q, k, v, g, offsets=off)
        grads = dw.linear_attention_grad(y, q, k, v, g, h0=hT, dhT=hT, offsets=off)
        one = dw.linear_attention_step(q[:5], k[:5], v[:5], g, h)
        n1, s1 = dw.group_norm(img, 12, w, w, act="silu", save_stats=True)
        n2, s2 = dw.group_norm(tok, 6, act="silu", save_stats=True)
        g1 = dw.group_norm_grad(dimg, img, s1, 12, w, w, act="silu")
        g2 = dw.group_norm_grad(dtok, tok, s2, 6, act="silu")
        p1 = dw.linear_i8(few, wq, ws, act="silu")
        p2 = dw.linear_i8(many, wq, ws)
        return [y, hT, *grads, one, h.clone(), n1, n2, *g1, *g2, p1, p2]

    return [q, k, v, img, tok, few, many, h], call


def test_same_bits_twice_and_on_another_stream(torch):
    for dtype in DTYPES:
        ins, call = _everything(torch, dtype)
        first = call()
        ins[-1].zero_()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            second = call()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, second))


def test_in_a_graph(torch):
    """A captured block, replayed with new inputs between eager calls."""
    for dtype in DTYPES:
        ins, call = _everything(torch, dtype)
        call()
        torch.cuda.synchronize()
        ins[-1].zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kept = call()
        for turn in range(3):
            rng = np.random.default_rng(100 + turn)
            for t in ins[:-1]:
                t.copy_(_gpu(torch, rng.standard_normal(t.shape)).to(t.dtype))
            ins[-1].zero_()
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in kept]
            ins[-1].zero_()
            want = call()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (dtype, turn)


def test_bad_offsets_stay_inside(torch):
    """Offsets that break the rules give unspecified rows, and no access outside."""
    rng = np.random.default_rng(1)
    q, k, v = (_draw(torch, rng, (300, 2, 64), "bfloat16")[0] for _ in range(3))
    g = torch.tensor([-0.01, -0.3], device="cuda")
    for off in ([0, 500, -7, 300], [0, 200, 100, 300], [5, 5, 5, 5], [0, 2 ** 31 - 1, -2 ** 31, 300]):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        y, h = dw.linear_attention(q, k, v, g, offsets=off)
        dw.linear_attention_grad(y, q, k, v, g, h0=h, dhT=h, offsets=off)
        torch.cuda.synchronize()
