"""The mixing operators at the ends of what their arguments may be."""
import pytest

import depthwise_convolution_amd as dw

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_quantize_the_longest_row(torch, dtype):
    """A row of 2^31 - 1 elements: its last ones, which fill no vector, lie less than a
    workgroup's threads before the end of 32-bit numbers."""
    K = (1 << 31) - 1
    x = torch.zeros(1, K, dtype=getattr(torch, dtype), device="cuda")
    q = torch.full((1, K), 99, dtype=torch.int8, device="cuda")
    scale = torch.empty(1, device="cuda")
    want = {0: 5, 1: -127, 4095: 2, K // 2: -64, K - 257: 1, K - 9: 126, K - 8: -1, K - 7: 7,
            K - 2: -3, K - 1: 127}
    for at, v in want.items():
        x[0, at] = v
    dw.dwconv_quantize_rows(x, q, scale)
    torch.cuda.synchronize()
    one = (torch.tensor(127.0) * torch.tensor(1 / 127)).item()     # in float32, as the header has it
    assert scale.item() == one
    for at, v in want.items():
        assert q[0, at].item() == v, at
    assert int((q != 0).sum()) == len(want)


def _norm_of_wide_rows(torch, P, C):
    """The forward and the gradient of one instance of P positions of C channels, in groups
    of 64, against float64 at both ends and around channel 2^30."""
    print(f"\n[case] norm of {P} x {C} channels", flush=True)
    torch.manual_seed(C % 1000)
    x, dy = (torch.empty(1, P, C, dtype=torch.bfloat16, device="cuda").uniform_(-2, 2)
             for _ in range(2))
    groups = C // 64
    y, stats = dw.group_norm(x, groups, save_stats=True)
    dx = torch.empty_like(x)
    gw, gb = (torch.full((C,), float("nan"), device="cuda") for _ in range(2))
    n = dw.dwconv_norm_workspace_size(True, x.dtype, 1, P, C, groups)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    dw.dwconv_norm_grad(dy, x, stats, groups, None, None, dx, gw, gb, workspace=ws)
    torch.cuda.synchronize()
    assert torch.isfinite(gw).all() and torch.isfinite(gb).all()
    wide = 64 * 64
    for lo in {0, min(1 << 30, C - wide) - wide // 2, C // 2 // 64 * 64, C - wide}:
        part = slice(lo, lo + wide)
        a, d = (t[0, :, part].double().unflatten(1, (-1, 64)) for t in (x, dy))
        mean = a.mean((0, 2), keepdim=True)
        rstd = 1 / (a.var((0, 2), unbiased=False, keepdim=True) + 1e-5).sqrt()
        xh = (a - mean) * rstd
        want = rstd * (d - d.mean((0, 2), keepdim=True) - xh * (d * xh).mean((0, 2), keepdim=True))
        # a few roundings of 64 * P numbers of at most 4, then the store's half step
        for got, ref, step in ((y[0, :, part], xh, 2.0 ** -8), (dx[0, :, part], want, 2.0 ** -8),
                               (gw[part], (d * xh).sum(0), 0.0), (gb[part], d.sum(0), 0.0)):
            ref = ref.reshape(got.shape)
            assert ((got.double() - ref).abs() <= 1e-4 + step * ref.abs()).all(), (lo, P)


@pytest.mark.parametrize("P", [1, 2])
def test_norm_of_more_than_2_30_channels(torch, P):
    """The 2 C sums of a gradient are more than 2^31."""
    _norm_of_wide_rows(torch, P, (1 << 30) + 128)


@pytest.mark.parametrize("P", [1, 2])
def test_norm_of_the_most_channels(torch, P):
    """A gradient takes as many workgroups as it needs, and not one for each channel."""
    _norm_of_wide_rows(torch, P, dw.SEQ_MAX_ROWS)


TOP = dw.SEQ_MAX_ROWS
PIECE = 1 << 27


def _pieces():
    return ((lo, min(lo + PIECE, TOP)) for lo in range(0, TOP, PIECE))


def _whole(torch, *shape):
    """Whole numbers from -3 to 3 in float16."""
    return torch.randint(-3, 4, shape, device="cuda", dtype=torch.int8).half()


def test_attention_of_the_most_rows(torch):
    """One sequence, and as many as rows: a head that forgets everything at once, so that
    each token stands for itself."""
    print(f"\n[case] linear_attention, one sequence of {TOP} tokens", flush=True)
    torch.manual_seed(1)
    q, k, v, dy = (_whole(torch, 1, TOP, 1, 1) for _ in range(4))
    g = torch.tensor([float("-inf")], device="cuda")
    y, hT = dw.linear_attention(q, k, v, g, scale=1.0)
    torch.cuda.synchronize()
    for lo, hi in _pieces():
        assert torch.equal(y[0, lo:hi], q[0, lo:hi] * k[0, lo:hi] * v[0, lo:hi]), lo
    assert hT.item() == (k[0, -1] * v[0, -1]).item()
    del y
    print("[case] its gradient", flush=True)
    dq, dk, dv, _ = dw.linear_attention_grad(dy, q, k, v, g, scale=1.0)
    torch.cuda.synchronize()
    for lo, hi in _pieces():
        a, b, c, d = (t[0, lo:hi] for t in (q, k, v, dy))
        assert torch.equal(dq[0, lo:hi], b * c * d), lo
        assert torch.equal(dk[0, lo:hi], c * d * a), lo
        assert torch.equal(dv[0, lo:hi], b * a * d), lo
    del dq, dk, dv
    print("[case] a token for each sequence", flush=True)
    h = torch.ones(TOP, 1, 1, 1, device="cuda")
    g = torch.zeros(1, device="cuda")
    y = dw.linear_attention_step(q[0], k[0], v[0], g, h, scale=1.0)
    torch.cuda.synchronize()
    for lo, hi in _pieces():
        state = 1 + k[0, lo:hi] * v[0, lo:hi]
        assert torch.equal(y[lo:hi], q[0, lo:hi] * state), lo
        assert torch.equal(h[lo:hi, 0], state.float()), lo


def test_norm_of_the_most_rows(torch):
    print(f"\n[case] group_norm of {TOP} tokens", flush=True)
    torch.manual_seed(2)
    x, dy = _whole(torch, TOP, 2), _whole(torch, TOP, 2)
    y, stats = dw.group_norm(x, 1, save_stats=True)
    dx, gw, gb = dw.group_norm_grad(dy, x, stats, 1)
    torch.cuda.synchronize()
    total = torch.zeros(2, dtype=torch.float64, device="cuda")
    for lo, hi in _pieces():
        a, d = x[lo:hi].double(), dy[lo:hi].double()
        half = (a[:, :1] - a[:, 1:]) / 2        # from the mean
        rstd = 1 / (half * half + 1e-5).sqrt()
        xh = torch.cat([half * rstd, -half * rstd], 1)
        want = rstd * (d - d.mean(1, True) - xh * (d * xh).mean(1, True))
        assert ((y[lo:hi].double() - xh).abs() <= 2.0 ** -10).all(), lo
        # where the two are equal rstd is 316 and half the difference of dy is its factor
        assert ((dx[lo:hi].double() - want).abs() <= 2.0 ** -10 * (want.abs() + 0.1)).all(), lo
        total += d.sum(0)
    # whole numbers of either sign: partial sums stay below 2^24, where float32 is exact
    assert torch.equal(gb.double(), total)


def test_products_of_the_most_rows(torch):
    print(f"\n[case] quantize_rows and linear_i8 of {TOP} rows", flush=True)
    torch.manual_seed(3)
    x = _whole(torch, TOP, 2)
    x[:, 0] = 127.0
    q, s = dw.quantize_rows(x)
    torch.cuda.synchronize()
    w = torch.tensor([[1, 2]], dtype=torch.int8, device="cuda")
    one = torch.ones(1, device="cuda")
    y = dw.linear_i8(q, w, one, x_scale=s, dtype=torch.float16)
    torch.cuda.synchronize()
    for lo, hi in _pieces():
        assert torch.equal(q[lo:hi], x[lo:hi].to(torch.int8)) and (s[lo:hi] == 1.0).all(), lo
        assert torch.equal(y[lo:hi, 0], x[lo:hi, 0] + 2 * x[lo:hi, 1]), lo
    del y
    y = dw.linear_i8(x, w, one)
    torch.cuda.synchronize()
    for lo, hi in _pieces():
        assert torch.equal(y[lo:hi, 0], x[lo:hi, 0] + 2 * x[lo:hi, 1]), lo


def test_norm_of_one_wide_group(torch):
    """A group of 2^27 channels: its workgroups do not each read all of its sums again, some
    2^43 bytes.  Every channel of half of them is 2, of the others -2."""
    C = 1 << 27
    x = torch.full((2, 2, C), 2.0, dtype=torch.bfloat16, device="cuda")
    x[..., C // 2:] = -2.0
    dy = torch.zeros_like(x)
    dy[0, :, :C // 4] = 8.0
    y, stats = dw.group_norm(x, 1, eps=0.0, save_stats=True)
    dx, gw, gb = dw.group_norm_grad(dy, x, stats, 1)
    torch.cuda.synchronize()
    # 2^16 workgroups' parts are joined by 256 threads and their tree: some 270 in a row, each
    # with two roundings of at most 2 and one of the mean, 270 * 3 * 2^-23 = 1e-4; the
    # variance alike, so that mean, rstd, and what follows from them by factors of up to 8
    # are within 1e-3, far below half a step of bfloat16's 1 and 2
    def near(t, want):
        return ((t.float() - want).abs() <= 1e-3).all()

    assert torch.equal(y, x / 2)
    assert near(stats[..., 0], 0.0) and near(stats[..., 1], 0.5)
    # instance 0: the means of dy and of dy * xhat are 8 / 4; dx = (dy - 2 - 2 xhat) / 2
    assert near(dx[1], 0.0)
    for lo, hi, want in ((0, C // 4, 2.0), (C // 4, C // 2, -2.0), (C // 2, C, 0.0)):
        assert near(dx[0, :, lo:hi], want)
    assert near(gw[:C // 4] / 16, 1.0) and (gb[:C // 4] == 16).all()
    assert not gw[C // 4:].any() and not gb[C // 4:].any()
