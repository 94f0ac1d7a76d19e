"""GPU parity of the mixing operators along the paths that only larger sizes take."""
import pytest

import depthwise_convolution_amd as dw

from . import sequence_gpu64 as on_gpu
from . import test_gpu_mixing as base
from .sequence_reference import EPS
from .test_gpu_mixing import DTYPES, torch  # noqa: F401

pytestmark = pytest.mark.gpu

# (shape, groups, act): groups that lie across the columns of two workgroups and more
WIDE_NORMS = [((2, 5, 20000), 8, "silu"), ((3, 70, 6144), 12, "none"), ((1, 40, 2304), 1, "relu"),
              ((2, 3, 4098), 6, "silu"), ((1, 9, 8192), 2048, "silu"),
              # and of more than 512 workgroups
              ((2, 3, 600000), 1, "silu"), ((2, 1200000), 2, "none"), ((3, 5, 2000), 2, "relu6")]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(WIDE_NORMS)))
def test_group_norm_across_columns(torch, monkeypatch, case, dtype):     # noqa: F811
    monkeypatch.setattr(base, "NORM_CASES", WIDE_NORMS)
    base.test_group_norm(torch, case, dtype)

# ------------------------------------------ matrix product in 8-bit integers
# (M, N, K, activation, bias, residual, aligned): which kernels these reach is checked,
# without a GPU, in tests/test_mixing_plans.py.  Rows behind the last tile's, columns that
# a vector of 4 or 8 does not end with, steps of k that are not full.
I8_LARGE = [
    (4099, 2049, 1040, "silu", True, True, True), (4098, 2052, 1040, "none", False, True, True),
    (1500, 2049, 16400, "relu", True, True, True), (2049, 4104, 528, "relu6", True, False, True),
    (4099, 770, 16400, "silu", True, True, True), (3001, 2049, 64, "relu6", True, True, True),
    (3001, 2049, 77, "silu", True, True, False), (1500, 2049, 16401, "none", True, True, False),
    (4097, 1031, 1040, "silu", False, True, False), (1029, 2049, 64, "silu", True, True, True),
    (65, 2049, 16400, "none", True, True, True), (1001, 2050, 61, "silu", True, True, False),
]


def i8_kernel_of(case, dtype):
    M, N, K, *_, aligned = case
    return dw.dwconv_linear_i8_describe(True, dtype, M, N, K, aligned=aligned)


def _int8(torch, gen, rows, K, aligned):        # noqa: F811
    """Rows of numbers from -127 to 127, on 16 bytes or 3 bytes behind, numbers between them."""
    pad = (K + 15) // 16 * 16 + 16 if aligned else K + 6
    wide = torch.randint(-127, 128, (rows, pad), generator=gen, device="cuda", dtype=torch.int8)
    return wide[:, :K] if aligned else wide[:, 3:3 + K]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(I8_LARGE)))
def test_linear_i8_large(torch, case, dtype):    # noqa: F811
    M, N, K, act, bias, res, aligned = spec = I8_LARGE[case]
    kind = getattr(torch, dtype)
    print(f"\n[case] linear_i8 {spec} {dtype} {i8_kernel_of(spec, kind)}", flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(case)

    def some(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    x, w = (_int8(torch, gen, rows, K, aligned) for rows in (M, N))
    xs, ws = (some(n) / 127 / K ** 0.25 / 64 for n in (M, N))
    b = some(N) - 0.5 if bias else None
    r = (some(M, N) - 0.5).to(kind) if res else None
    y = torch.full((M + 2, N + 3), 7.0, dtype=kind, device="cuda")
    n = dw.dwconv_linear_i8_workspace_size(torch.int8, kind, M, N, K)
    space = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    dw.dwconv_linear_i8(x, w, ws, b, y[1:-1, 2:-1], act=act, res=r, x_scale=xs, workspace=space)
    torch.cuda.synchronize()
    # the sums are whole numbers, which float64 holds; the scales, their product and its
    # product with the sum are rounded, and what is added to it
    z0 = (x.double() @ w.double().T) * xs.double()[:, None] * ws.double()
    z = z0 + b.double() if bias else z0
    z_err = 4 * EPS * z0.abs() + EPS * z.abs()
    # an activation's slope is below 1.1, its own error as in tests/sequence_reference.py
    want = on_gpu.act(z, act)
    tol = 1.1 * z_err + (EPS * (8 + 2 * z.abs()) * want.abs() if act == "silu" else 0.0)
    if res:
        want = want + r.double()
        tol = tol + EPS * want.abs()
    on_gpu.near(y[1:-1, 2:-1], want, on_gpu.store_tol(want, tol, dtype), "y")
    y[1:-1, 2:-1] = 7.0
    assert (y == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_i8_quantises_for_the_large_tiles(torch, dtype):      # noqa: F811
    """x in a float type gives the bits that its numbers made beforehand give."""
    kind = getattr(torch, dtype)
    for M, N, K in ((4099, 2049, 1040), (3001, 2049, 77)):
        x = torch.randn(M, K, device="cuda").to(kind)
        wq, ws = dw.quantize_rows(torch.randn(N, K, device="cuda"))
        q, s = dw.quantize_rows(x)
        assert torch.equal(dw.linear_i8(x, wq, ws, act="silu"),
                           dw.linear_i8(q, wq, ws, act="silu", x_scale=s, dtype=kind))


# --------------------------------------------- statistics joined by a launch of their own
# more than 128 ranges of rows
JOINED_NORMS = [((1, 97, 91, 256), 32, "silu"), ((1, 9001, 260), 4, "relu"),
                ((2, 190, 180, 64), 1, "none"), ((1, 310, 300, 24), 24, "silu")]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(JOINED_NORMS)))
def test_group_norm_of_many_ranges(torch, monkeypatch, case, dtype):      # noqa: F811
    shape, groups, act = JOINED_NORMS[case]
    monkeypatch.setattr(base, "NORM_CASES", JOINED_NORMS)
    base.test_group_norm(torch, case, dtype)
    # in place, without statistics kept
    x, w, b, *_ = base._norm_inputs(torch, JOINED_NORMS[case], dtype, case)
    want = dw.group_norm(x, groups, w, b, act=act)
    P = x.numel() // x.shape[0] // x.shape[-1]
    n = dw.dwconv_norm_workspace_size(False, x.dtype, x.shape[0], P, x.shape[-1], groups)
    space = torch.empty(n, dtype=torch.uint8, device="cuda")
    dw.dwconv_norm_fwd(x, groups, w, b, x, act=act, workspace=space)
    assert torch.equal(x, want)


def _filled(torch, n, value):        # noqa: F811
    return torch.full((n,), value, dtype=torch.uint8, device="cuda") if n else None


@pytest.mark.parametrize("dtype", DTYPES)
def test_what_a_workspace_held_before_does_not_matter(torch, dtype):     # noqa: F811
    kind = getattr(torch, dtype)
    for shape, groups in ((s[0], s[1]) for s in WIDE_NORMS + JOINED_NORMS):
        N, C = shape[0], shape[-1]
        x, dy = (torch.randn(shape, device="cuda").to(kind) for _ in range(2))
        P = x.numel() // N // C
        sizes = [dw.dwconv_norm_workspace_size(g, kind, N, P, C, groups) for g in (False, True)]
        got = []
        for value in (0, 255):
            y, dx = torch.empty_like(x), torch.empty_like(x)
            stats = torch.empty(N, groups, 2, device="cuda")
            gw, gb = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
            dw.dwconv_norm_fwd(x, groups, None, None, y, act="silu", stats=stats,
                               workspace=_filled(torch, sizes[0], value))
            dw.dwconv_norm_grad(dy, x, stats, groups, None, None, dx, gw, gb, act="silu",
                                workspace=_filled(torch, sizes[1], value))
            got.append((y, stats, dx, gw, gb))
        assert all(torch.equal(a, b) for a, b in zip(*got)), (shape, groups)
    for M, N, K, *_ in I8_LARGE[:3] + I8_LARGE[10:] + [(8, 256, 512), (40, 100, 8192)]:
        x = torch.randn(M, K, device="cuda").to(kind)
        w, s = dw.quantize_rows(torch.randn(N, K, device="cuda"))
        n = dw.dwconv_linear_i8_workspace_size(kind, kind, M, N, K)
        got = []
        for value in (0, 255):
            y = torch.empty(M, N, dtype=kind, device="cuda")
            got.append(dw.dwconv_linear_i8(x, w, s, None, y, workspace=_filled(torch, n, value)))
        assert torch.equal(*got), (M, N, K)
