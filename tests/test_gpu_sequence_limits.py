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
