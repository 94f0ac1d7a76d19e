"""The sequence operators at the most rows they accept, where 32-bit row numbers
have little room left, and past 2^32 elements.  Everything of one or few channels,
checked on the device in pieces."""
import pytest

import depthwise_convolution_amd as dw

pytestmark = pytest.mark.gpu

TOP = dw.SEQ_MAX_ROWS
PIECE = 1 << 27


@pytest.fixture(scope="module")
def torch():
    import torch as t
    if not t.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    return t


@pytest.fixture(autouse=True)
def _free():
    yield
    import torch as t
    if t.cuda.is_available():
        t.cuda.empty_cache()


def _whole(torch, gen, *shape):
    """Whole numbers from -3 to 3 in float16."""
    return torch.randint(-3, 4, shape, generator=gen, device="cuda", dtype=torch.int8).half()


def _gen(torch):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    return gen


def test_causal_conv_of_the_most_rows(torch):
    print(f"\n[case] causal_conv {TOP} rows", flush=True)
    gen = _gen(torch)
    x, dy = _whole(torch, gen, 1, TOP, 1), _whole(torch, gen, 1, TOP, 1)
    w = torch.tensor([[2.0, -1.0, 3.0]], device="cuda")
    y = torch.full_like(x, float("nan"))
    dw.dwconv_causal_fwd(x, w, None, y)
    torch.cuda.synchronize()
    print("[case] its gradient", flush=True)
    dx, dW, db, _ = dw.causal_conv_grad(dy, x, w)
    torch.cuda.synchronize()
    taps = w[0].half()
    sums, total = [0, 0, 0], 0
    for lo in range(0, TOP, PIECE):
        hi = min(lo + PIECE, TOP)
        want, grad = torch.zeros_like(x[0, lo:hi, 0]), torch.zeros_like(x[0, lo:hi, 0])
        total += int(dy[0, lo:hi, 0].sum(dtype=torch.float64))
        for j in range(3):
            back = 2 - j
            start = max(lo - back, 0)
            row = x[0, start:hi - back, 0]
            want[hi - lo - len(row):] += taps[j] * row
            sums[j] += int((row.double() * dy[0, hi - len(row):hi, 0]).sum())
            row = dy[0, lo + back:hi + back, 0]
            grad[:len(row)] += taps[j] * row
        assert torch.equal(y[0, lo:hi, 0], want), lo
        assert torch.equal(dx[0, lo:hi, 0], grad), lo
    # sums of 2^31 numbers up to 9: float32 additions in chains of some 2^20 rows and
    # shorter ones, each off by 2^-24 of what it has reached, which a random walk
    # of whole numbers keeps below 2^24 -- where they are exact
    for got, exact in zip([float(v) for v in dW[0]] + [float(db)], [*sums, total]):
        assert abs(got - exact) <= 2.0 ** -20 * abs(exact) + 1, (got, exact)


def test_causal_conv_of_many_sequences(torch):
    """More than 2^30 sequences, all but the last of no token."""
    seqs, n, C = (1 << 30) + 9, 1000, 8
    print(f"\n[case] causal_conv {seqs} sequences", flush=True)
    gen = _gen(torch)
    x = _whole(torch, gen, n, C)
    w = torch.randint(-2, 3, (C, 4), generator=gen, device="cuda").float()
    offsets = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = n
    y = dw.dwconv_causal_fwd(x, w, None, torch.full_like(x, float("nan")), offsets=offsets)
    want, _ = dw.causal_conv(x[None], w)
    torch.cuda.synchronize()
    assert torch.equal(y, want[0])


def test_linear_gradient_over_the_most_rows(torch):
    """dz, dw and db, where the rows are the summed index: a few rows that are
    not zero, the last ones among them."""
    print(f"\n[case] linear_grad over {TOP} rows", flush=True)
    x = torch.zeros(TOP, 1, dtype=torch.float16, device="cuda")
    dy, z = torch.zeros_like(x), torch.zeros_like(x)
    w = torch.ones(1, 1, dtype=torch.float16, device="cuda")
    at = torch.tensor([0, 1, PIECE, TOP // 2, TOP - 65, TOP - 9, TOP - 2, TOP - 1], device="cuda")
    x[at, 0] = torch.arange(1.0, 9.0, device="cuda").half()
    dy[at, 0] = 2.0 ** torch.arange(8.0, device="cuda").half()
    z[at, 0] = 1.0
    z[TOP - 2] = -1.0           # ReLU: not this one
    dW = torch.empty(1, 1, dtype=torch.float16, device="cuda")
    db = torch.empty(1, device="cuda")
    space = torch.empty(dw.dwconv_linear_workspace_size(True, x.dtype, "relu", TOP, 1, 1),
                        dtype=torch.uint8, device="cuda")
    dw.dwconv_linear_grad(dy, x, w, None, dW, db, z=z, workspace=space, act="relu")
    torch.cuda.synchronize()
    kept = [0, 1, 2, 3, 4, 5, 7]
    assert float(db) == sum(2.0 ** k for k in kept)
    assert float(dW) == sum(2.0 ** k * (k + 1) for k in kept)
    dw.dwconv_linear_grad(dy, x, w, None, dW, db, workspace=space)
    torch.cuda.synchronize()
    assert float(db) == 255.0 and float(dW) == sum(2.0 ** k * (k + 1) for k in range(8))


def test_causal_conv_past_2_to_32_elements(torch):
    """4.3e9 elements: the last sequence equals a call of its own."""
    seqs, T, C = 1030, 1024, 4096
    print(f"\n[case] causal_conv {seqs} x {T} x {C}", flush=True)
    gen = _gen(torch)
    x = torch.empty(seqs, T, C, dtype=torch.bfloat16, device="cuda")
    for k in range(0, seqs, 103):
        x[k:k + 103].normal_(generator=gen)
    w = torch.randn(C, 4, generator=gen, device="cuda")
    y, final = dw.causal_conv(x, w, act="silu")
    dx = dw.causal_conv_grad(x, x, w, act="silu")[0]
    for k in (0, 511, 1023, 1024, seqs - 1):
        mine = x[k:k + 1].clone()
        want, last = dw.causal_conv(mine, w, act="silu")
        grad = dw.causal_conv_grad(mine, mine, w, act="silu")[0]
        torch.cuda.synchronize()
        assert torch.equal(y[k], want[0]) and torch.equal(final[k], last[0]), k
        assert torch.equal(dx[k], grad[0]), k


# ------------------- more than 2^32 threads, which a grid of one dimension does not hold
def _gates(torch, gen, *shape):
    return [torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16)
            for _ in range(3)]


def test_scan_of_many_short_sequences(torch):
    """A workgroup for each sequence: 4.2 million of one token and 3 channels have
    more than 2^32 threads.  The first and last ones equal calls of their own."""
    seqs, C = (1 << 22) + 5, 3
    print(f"\n[case] gated_scan {seqs} x 1 x {C}", flush=True)
    gen = _gen(torch)
    x, r, i = _gates(torch, gen, seqs, 1, C)
    lam = torch.tensor([-3.0, 0.0, 2.0], device="cuda")
    h0, dhT = torch.randn(2, seqs, C, generator=gen, device="cuda")
    y, hT, states = dw.gated_scan(x, r, i, lam, h0=h0, save_states=True)
    dx, dr, di, dlam, dh0 = dw.gated_scan_grad(x, x, r, i, lam, states, dhT=dhT)
    torch.cuda.synchronize()
    shares = torch.zeros(C, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(shares)
    for lo in range(0, seqs, 1 << 20):
        k = slice(lo, min(lo + (1 << 20), seqs))
        want, last, kept = dw.gated_scan(x[k], r[k], i[k], lam, h0=h0[k], save_states=True)
        grads = dw.gated_scan_grad(x[k], x[k], r[k], i[k], lam, kept, dhT=dhT[k])
        torch.cuda.synchronize()
        for a, b in zip((y, hT, dx, dr, di, dh0), (want, last, *grads[:3], grads[4])):
            assert torch.equal(a[k], b), lo
        shares += grads[3].double()
        size += grads[3].double().abs()
    # some 2^18 additions in a row at most, of shares of either sign
    assert bool(((dlam.double() - shares).abs() <= 2.0 ** -12 * size.clamp(min=1e3)).all())


def test_scan_of_the_most_rows(torch):
    """One sequence: a chain of 2^24 runs.  Its memory is short, so the last tokens
    equal a call that begins some thousand before."""
    print(f"\n[case] gated_scan {TOP} rows", flush=True)
    gen = _gen(torch)
    x = torch.empty(1, TOP, 1, dtype=torch.float16, device="cuda")
    for lo in range(0, TOP, PIECE):
        x[0, lo:lo + PIECE].normal_(generator=gen)
    lam = torch.tensor([0.0], device="cuda")        # a = e^(-5.5 sigmoid(r))
    y, hT = dw.gated_scan(x, x, x, lam)
    torch.cuda.synchronize()
    for lo, hi in ((0, 5000), (PIECE, PIECE + 5000), (TOP - 5000, TOP)):
        part = x[:, lo:hi]
        want, last = dw.gated_scan(part, part, part, lam)
        torch.cuda.synchronize()
        off = (y[0, lo + 2000:hi, 0].double() - want[0, 2000:, 0].double()).abs()
        # float16 results of float32 states of up to some 4, a few roundings apart: the
        # next number at most
        tol = 2.0 ** -10 * want[0, 2000:, 0].double().abs() + 2.0 ** -20
        assert bool((off <= tol).all()), lo
    assert abs(float(hT) - float(last)) <= 2.0 ** -18 * abs(float(last)) + 1e-6
    assert bool(torch.isfinite(y).all())


def test_chained_scan_of_many_sequences(torch):
    """Linked runs: a million sequences of one token, then one of a thousand."""
    seqs, C, last = 1 << 20, 1024, 1000
    print(f"\n[case] gated_scan {seqs} + {last} rows x {C}, packed", flush=True)
    gen = _gen(torch)
    n = seqs - 1 + last
    x = torch.empty(n, C, dtype=torch.bfloat16, device="cuda")
    for lo in range(0, n, 1 << 17):
        x[lo:lo + (1 << 17)].normal_(generator=gen)
    lam = torch.randn(C, generator=gen, device="cuda") - 4
    offsets = torch.arange(seqs + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = n
    y, hT = dw.gated_scan(x, x, x, lam, offsets=offsets)
    torch.cuda.synchronize()
    for lo in (0, 1 << 19, seqs - 1 - 4096):
        part = x[lo:lo + 4096, None]
        want, ends = dw.gated_scan(part, part, part, lam)
        torch.cuda.synchronize()
        assert torch.equal(y[lo:lo + 4096], want[:, 0]) and torch.equal(hT[lo:lo + 4096], ends)
    part = x[None, seqs - 1:]
    want, ends = dw.gated_scan(part, part, part, lam)
    torch.cuda.synchronize()
    assert torch.equal(y[seqs - 1:], want[0]) and torch.equal(hT[-1:], ends)


def test_steps_of_many_sequences(torch):
    seqs, C = 1_440_000_000, 3
    print(f"\n[case] causal_conv_step {seqs} x {C}", flush=True)
    gen = _gen(torch)
    x = torch.empty(seqs, C, dtype=torch.float16, device="cuda")
    state = torch.empty(seqs, 1, C, dtype=torch.float16, device="cuda")
    for lo in range(0, seqs, PIECE):
        x[lo:lo + PIECE] = _whole(torch, gen, min(PIECE, seqs - lo), C)
        state[lo:lo + PIECE, 0] = x[lo:lo + PIECE].flip(1)
    w = torch.tensor([[1.0, 2.0], [-1.0, 3.0], [2.0, 0.0]], device="cuda")
    y = dw.causal_conv_step(x, state, w)
    torch.cuda.synchronize()
    for lo in range(0, seqs, PIECE):
        k = slice(lo, lo + PIECE)
        taps = w.half()
        assert torch.equal(y[k], taps[:, 0] * x[k].flip(1) + taps[:, 1] * x[k]), lo
        assert torch.equal(state[k, 0], x[k]), lo
    del state
    print(f"[case] gated_scan_step {seqs} x {C}", flush=True)
    lam = torch.tensor([-3.0, 0.0, 2.0], device="cuda")
    h = torch.ones(seqs, C, device="cuda")
    y = dw.dwconv_scan_step(x, x, x, lam, h, y)
    torch.cuda.synchronize()
    for lo in range(0, seqs, PIECE):
        k = slice(lo, lo + PIECE)
        mine = torch.ones_like(h[k])
        want = dw.gated_scan_step(x[k], x[k], x[k], lam, mine)
        torch.cuda.synchronize()
        assert torch.equal(y[k], want) and torch.equal(h[k], mine), lo


def test_carried_rows_of_many_sequences(torch):
    """4.3e9 elements of final and dinit: of one token each, after 7 carried rows."""
    seqs, C, K = 205_000_000, 3, 8
    print(f"\n[case] causal_conv carried rows {seqs} x {K - 1} x {C}", flush=True)
    gen = _gen(torch)
    x = _whole(torch, gen, seqs, 1, C)
    init = torch.empty(seqs, K - 1, C, dtype=torch.float16, device="cuda")
    for j in range(K - 1):
        init[:, j] = x[:, 0] + j
    w = torch.arange(1.0, 1.0 + C * K, device="cuda").view(C, K) % 5 - 2
    y, final = dw.causal_conv(x, w, init=init)
    dx, _, _, dinit = dw.causal_conv_grad(x, x, w, init=init)
    torch.cuda.synchronize()
    taps = w.half()
    for lo in range(0, seqs, 1 << 25):
        k = slice(lo, lo + (1 << 25))
        row = x[k, 0]
        z = taps[:, K - 1] * row
        for j in range(K - 1):
            z += taps[:, j] * init[k, j]
            assert torch.equal(dinit[k, j], taps[:, j] * row), (lo, j)
            assert torch.equal(final[k, j], init[k, j + 1] if j < K - 2 else row), (lo, j)
        assert torch.equal(y[k, 0], z) and torch.equal(dx[k, 0], taps[:, K - 1] * row), lo


def test_linear_over_the_most_rows(torch):
    print(f"\n[case] linear and its dx over {TOP} rows", flush=True)
    gen = _gen(torch)
    x = torch.empty(TOP, 1, dtype=torch.float16, device="cuda")
    for lo in range(0, TOP, PIECE):
        x[lo:lo + PIECE] = _whole(torch, gen, min(PIECE, TOP - lo), 1)
    w = torch.full((1, 1), -2.0, dtype=torch.float16, device="cuda")
    y = dw.linear(x, w, act="relu")
    dx = torch.full_like(x, float("nan"))
    space = torch.empty(dw.dwconv_linear_workspace_size(True, x.dtype, "none", TOP, 1, 1),
                        dtype=torch.uint8, device="cuda")
    dw.dwconv_linear_grad(x, x, w, dx, None, None, workspace=space)
    torch.cuda.synchronize()
    for lo in range(0, TOP, PIECE):
        k = slice(lo, lo + PIECE)
        assert torch.equal(y[k], (-2.0 * x[k]).clamp(min=0)), lo
        assert torch.equal(dx[k], -2.0 * x[k]), lo
