"""GPU parity of the mixing operators along the paths that only larger sizes take."""
import pytest

from . import test_gpu_mixing as base
from .test_gpu_mixing import DTYPES, torch  # noqa: F401

pytestmark = pytest.mark.gpu

# (shape, groups, act): groups that lie across the columns of two workgroups and more
WIDE_NORMS = [((2, 5, 20000), 8, "silu"), ((3, 70, 6144), 12, "none"), ((1, 40, 2304), 1, "relu"),
              ((2, 3, 4098), 6, "silu"), ((1, 9, 8192), 2048, "silu")]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(WIDE_NORMS)))
def test_group_norm_across_columns(torch, monkeypatch, case, dtype):     # noqa: F811
    monkeypatch.setattr(base, "NORM_CASES", WIDE_NORMS)
    base.test_group_norm(torch, case, dtype)
