"""Workspaces of the mixing operators where there are many groups or sequences, without a
GPU."""
import torch

import depthwise_convolution_amd as dw


def test_norm_workspace_counts_the_columns_that_a_group_lies_in():
    """Statistics of each range of rows for each group, and no room for the workgroups'
    columns that the group does not touch: at most two of them for narrow groups."""
    for C, groups in ((1 << 16, 1 << 16), (1 << 20, 1 << 14), (5000 * 64, 5000), (20000, 8)):
        for dtype in (torch.float32, torch.bfloat16):
            n = dw.dwconv_norm_workspace_size(False, dtype, 1, 2, C, groups)     # one range
            block = 256 if dtype is torch.float32 else 512      # columns of 256 vectors, at least
            wide = min(-(-C // groups) // block + 2, -(-C // block))
            assert 0 < n <= 8 * groups * wide + 16, (C, groups, dtype)
