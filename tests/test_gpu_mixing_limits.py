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
