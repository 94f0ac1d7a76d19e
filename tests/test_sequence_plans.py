"""Which kernels the large parity cases of the matrix product reach, without a
GPU: all tiles, in every order of the operands, along both paths to LDS, whole
and split.  A change of the cost model that loses one fails here."""
import pytest

import depthwise_convolution_amd as dw

from .test_gpu_linear_large import LINEAR_CASES, kernels_of

WIDE = {("y", "tile_256", False), ("y", "tile_256", True), ("dx", "tile_256", False),
        ("dx", "tile_256", True), ("dw", "tile_256", False),
        ("y", "tile_128", False), ("y", "tile_128", True), ("dx", "tile_128", False),
        ("dx", "tile_128", True), ("dw", "tile_128", False), ("dw", "tile_128", True),
        ("y", "tile_128_registers", False), ("dx", "tile_128_registers", False),
        ("dw", "tile_128_registers", False)}
NARROW = {("y", "tile_128", False), ("dx", "tile_128", False), ("dx", "tile_128", True),
          ("dw", "tile_128", False), ("y", "tile_128_registers", False),
          ("dx", "tile_128_registers", False), ("dw", "tile_128_registers", False),
          ("y", "tile_64", False), ("y", "tile_64", True), ("dx", "tile_64", False),
          ("dx", "tile_64", True), ("dw", "tile_64", False), ("dw", "tile_64", True)}


@pytest.mark.parametrize("dtype,size,want", [("bfloat16", 2, WIDE), ("float16", 2, WIDE),
                                             ("float32", 4, NARROW)])
def test_large_cases_reach_the_kernels(dtype, size, want):
    import torch
    got = set()
    for case in LINEAR_CASES:
        for product, (kernel, splits) in kernels_of(case, getattr(torch, dtype), size).items():
            got.add((product, kernel, splits > 1))
    assert want <= got, sorted(want - got)


def test_describe():
    import torch
    kind = torch.bfloat16
    assert dw.dwconv_linear_describe(dw.LINEAR_Y, kind, 8, 8192, 2048) == ("few_rows", 1)
    # K of an odd width is never read straight to LDS along k, and always across it
    assert dw.dwconv_linear_describe(dw.LINEAR_Y, kind, 300, 700, 901)[0].endswith("registers")
    assert not dw.dwconv_linear_describe(dw.LINEAR_DW, kind, 300, 700, 901)[0].endswith("registers")
    for args in ((3, kind, 8, 8, 8), (-1, kind, 8, 8, 8)):
        with pytest.raises(dw.DwconvError, match="BAD_OP|op"):
            dw.dwconv_linear_describe(*args)
    for args in ((0, torch.int32, 8, 8, 8), (0, kind, -1, 8, 8), (1, kind, 8, 0, 8),
                 (2, kind, 8, 8, 0)):
        with pytest.raises(dw.DwconvError):
            dw.dwconv_linear_describe(*args)
