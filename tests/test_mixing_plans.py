"""Which kernels the large parity cases of the mixing operators reach, without a GPU.  A
change of a plan that loses one fails here."""
import pytest
import torch

import depthwise_convolution_amd as dw

from .test_gpu_mixing import I8_CASES
from .test_gpu_mixing_paths import I8_LARGE, JOINED_NORMS, i8_kernel_of

TILES = {("tile_256", False), ("tile_256", True), ("tile_128", False), ("tile_128", True),
         ("tile_128_registers", False), ("tile_128_registers", True), ("tile_64", False),
         ("tile_64", True), ("tile_64_registers", False), ("tile_64_registers", True),
         ("tile_64_deep", False), ("tile_64_deep", True), ("few_rows", False),
         ("few_rows_quantized", False)}


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_cases_reach_the_kernels(dtype):
    got = {i8_kernel_of(case, dtype) for case in I8_LARGE}
    for M, N, K, *_ in I8_CASES:
        got |= {dw.dwconv_linear_i8_describe(False, dtype, M, N, K, aligned=K % 16 == 0),
                dw.dwconv_linear_i8_describe(True, dtype, M, N, K, aligned=K % 16 == 0),
                dw.dwconv_linear_i8_describe(True, dtype, M, N, K, aligned=False)}
    got = {(kernel, splits > 1) for kernel, splits in got}
    assert TILES <= got, sorted(TILES - got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_many_ranges(dtype):
    """The statistics of more than 128 ranges are joined by a launch of their own, into
    2 float32 a group behind the ranges' in the workspace."""
    for shape, groups, _ in JOINED_NORMS:
        N, C, P = shape[0], shape[-1], 1
        for n in shape[1:-1]:
            P *= n
        sizes = dw.dwconv_norm_workspace_size(False, dtype, N, P, C, groups)
        assert sizes > 8 * N * groups * 129, (shape, dtype)
