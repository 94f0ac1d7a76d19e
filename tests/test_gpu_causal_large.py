"""GPU parity of the causal convolution at sizes where a thread walks many rows,
against float64 on the device (tests/sequence_gpu64.py), mostly on small whole
numbers, whose sums are exact; and single tokens of all sequence operators in a graph.
"""
import numpy as np
import pytest

import depthwise_convolution_amd as dw

from .sequence_reference import EPS

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


# ------------------------------------------- causal depthwise convolution
def _cuts(rng, rows, seqs, K):
    """Offsets of a ragged batch: sequences of no token, of one, shorter than the
    filter, and cuts one after the other inside a thread's rows."""
    cuts = np.sort(rng.integers(0, rows + 1, seqs - 1))
    cuts[1] = cuts[0]
    for k in range(5, min(5 + K, len(cuts))):
        cuts[k] = min(cuts[4] + k - 4, rows)
    cuts = np.sort(cuts)
    return np.concatenate([[0], cuts, [rows]]).astype(np.int32)


# Large enough for the longest walks: 32 rows a thread in the forward (33.5M
# elements), 64 in the gradient (16.8M), 256 where there are more rows
CONV_CASES = [
    # (rows or (S, T), sequences, C, K, activation, carry, strided)
    ((5, 13001), None, 520, 4, "relu", True, False),
    (300007, 401, 130, 3, "none", True, True),
    ((3, 22001), None, 528, 8, "none", False, True),
    (70003, 57, 512, 4, "silu", False, False),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(CONV_CASES)))
def test_causal_conv_large(torch, ref, case, dtype):
    layout, seqs, C, K, act, carry, strided = spec = CONV_CASES[case]
    print(f"\n[case] large causal_conv {spec} {dtype}", flush=True)
    rng = np.random.default_rng(case)
    if seqs is None:
        seqs, offsets = layout[0], np.arange(layout[0] + 1) * layout[1]
        shape, off = (*layout, C), None
    else:
        offsets = _cuts(rng, layout, seqs, K)
        shape, off = (layout, C), torch.from_numpy(offsets).cuda()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(case)
    whole = act != "silu"       # whole numbers: every sum is exact

    def draw(shape, top, kind):
        if whole:
            t = torch.randint(-top, top + 1, shape, generator=gen, device="cuda")
        else:
            t = torch.randn(shape, generator=gen, device="cuda")
        return t.to(getattr(torch, kind))

    x, dy = draw(shape, 3, dtype), draw(shape, 3, dtype)
    w, b = draw((C, K), 2, "float32"), draw((C,), 2, "float32")
    init = draw((seqs, K - 1, C), 3, dtype) if carry else None
    dfinal = draw((seqs, K - 1, C), 3, dtype) if carry else None
    if strided:
        x, dy = (torch.cat([t[..., :5], t, t[..., :3]], -1)[..., 5:5 + C] for t in (x, dy))
    y, final = dw.causal_conv(x, w, b, act=act, init=init, offsets=off)
    got = dw.causal_conv_grad(dy, x, w, b, act=act, init=init, offsets=off)
    ends = dw.causal_conv_grad(dy, x, w, b, act=act, init=init, dfinal=dfinal, offsets=off)
    torch.cuda.synchronize()
    rows = ref.Rows(offsets)
    xd, dyd = x.double().reshape(-1, C), dy.double().reshape(-1, C)
    wd, bd, initd = w.double(), b.double(), None if init is None else init.double()
    z = ref.conv(xd, wd, bd, rows, initd)
    assert torch.equal(final.double(), ref.conv_final(xd, K, rows, initd))
    want = ref.act(z, act)
    dz = dyd * ref.slope(z, act)
    dx, dW, db = ref.conv_grad(dz, xd, wd, rows, initd)
    if whole:
        assert torch.equal(y.double().reshape(-1, C), want)
        for name, t, v in zip(("dx", "dw", "db"), got, (dx, dW, db)):
            assert torch.equal(t.double().reshape(v.shape), v), name
        if carry:
            # dfinal reaches the last K-1 rows, and where a sequence is shorter than that, dinit
            tail = dx.clone()
            short = dfinal.double()
            for j in range(K - 1):
                at = rows.end - (K - 1) + j
                inside = at >= rows.start
                tail.index_put_((at[inside],), short[inside, j], accumulate=True)
            assert torch.equal(ends[0].double().reshape(-1, C), tail)
            assert torch.equal(ends[1], got[1]) and torch.equal(ends[2], got[2])
        return
    # as in the tests of small sizes, with the number of roundings in a row of
    # the sums as they are taken: a thread's rows, 4 threads, 16 sums by turns
    big = ref.conv(xd.abs(), wd.abs(), bd.abs(), rows, None)
    tol = 1.1 * (K + 2) * EPS * big + EPS * (8 + 2 * z.abs()) * want.abs()
    ref.near(y, want, ref.store_tol(want, tol, dtype), "y")
    top = float(big.max())
    c = (24 + 4 * top + K + 0.5 * (K + 2) * top) * EPS
    majorants = ref.conv_grad(dyd.abs(), xd.abs(), wd.abs(), rows, None)
    for name, t, v, m, n, kind in zip(("dx", "dw", "db"), got, (dx, dW, db), majorants,
                                      (K, 128, 128), (dtype, "float32", "float32")):
        ref.near(t, v, ref.store_tol(v, (c + n * EPS) * m * 1.1 + 1e-30, kind), name)


# ------------------------------------------------------------ single tokens in a graph
def test_steps_in_a_graph(torch):
    """One token of each sequence through all three operators, captured once and
    replayed, the states carried on from replay to replay, eager work between."""
    S, C, H, K = 7, 40, 72, 4
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)

    def draw(*shape, kind=torch.bfloat16):
        return torch.randn(shape, generator=gen, device="cuda").to(kind)

    x = draw(S, C)
    w_in, w_gate, w_out = draw(H, C) / 6, draw(2 * H, H) / 8, draw(C, H) / 8
    w_conv, lam = draw(H, K, kind=torch.float32) / 2, draw(H, kind=torch.float32) - 4

    def step(rows, h):
        u = dw.linear(x, w_in)
        v = dw.causal_conv_step(u, rows, w_conv, act="silu")
        r, i = dw.linear(v, w_gate).chunk(2, dim=-1)
        y = dw.gated_scan_step(v, r, i, lam, h)
        return dw.linear(y, w_out, res=x)

    def fresh():
        return torch.zeros(S, K - 1, H, dtype=torch.bfloat16, device="cuda"), \
            torch.zeros(S, H, device="cuda")

    tokens = [draw(S, C) for _ in range(5)]
    rows, h = fresh()
    want = []
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for t in tokens:
            x.copy_(t)
            want.append(step(rows, h).clone())
    side.synchronize()
    last = rows.clone(), h.clone()
    rows, h = fresh()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = step(rows, h)
    for k, t in enumerate(tokens):
        x.copy_(t)
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[k]), f"token {k}"
        with torch.cuda.stream(side):
            step(*fresh())
        side.synchronize()
    assert torch.equal(rows, last[0]) and torch.equal(h, last[1])
