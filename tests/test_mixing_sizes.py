"""Workspaces of the mixing operators where there are many groups or sequences, without a
GPU."""
import pytest
import torch

import depthwise_convolution_amd as dw
from depthwise_convolution_amd import sequence

from .test_sequence_devices import OnGpu


def test_norm_workspace_counts_the_columns_that_a_group_lies_in():
    """Statistics of each range of rows for each group, and no room for the workgroups'
    columns that the group does not touch: at most two of them for narrow groups."""
    for C, groups in ((1 << 16, 1 << 16), (1 << 20, 1 << 14), (5000 * 64, 5000), (20000, 8)):
        for dtype in (torch.float32, torch.bfloat16):
            n = dw.dwconv_norm_workspace_size(False, dtype, 1, 2, C, groups)     # one range
            block = 256 if dtype is torch.float32 else 512      # columns of 256 vectors, at least
            wide = min(-(-C // groups) // block + 2, -(-C // block))
            assert 0 < n <= 8 * groups * wide + 16, (C, groups, dtype)


class Dense(OnGpu):
    def is_contiguous(self):
        return True


def _far(*shape, dtype=torch.float32):
    """A stand-in on a GPU with that shape, all of it one element."""
    return torch.zeros(1, dtype=dtype).expand(*shape).as_subclass(Dense)


BIG = (1 << 32) + 4        # 4 in 32 bits


def test_axes_that_32_bits_do_not_hold_are_refused(monkeypatch):
    """An axis is passed on in 32 bits; one of 2^32 + 4 is not taken as 4, nor as none where
    nothing else is."""
    sequence._setup()
    monkeypatch.setattr(sequence, "_raw_stream", lambda index: 0)
    q, x, g = _far(1, 1, 4, 8), _far(2, 8), _far(4)
    off = _far(BIG + 1, dtype=torch.int32)
    w8 = _far(BIG, 8, dtype=torch.int8)
    taps = _far(8, BIG)
    calls = {
        "heads": lambda: dw.linear_attention(_far(1, 1, BIG, 8), q, q, g),
        "width": lambda: dw.linear_attention(q, q, _far(1, 1, 4, BIG), g),
        "sequences": lambda: dw.linear_attention_step(*[_far(BIG, 4, 8)] * 3, g, g),
        "gradient": lambda: dw.linear_attention_grad(q, *[_far(BIG, 1, 4, 8)] * 3, g),
        "offsets": lambda: dw.linear_attention(*[_far(5, 4, 8)] * 3, g, offsets=off),
        "channels": lambda: dw.group_norm(_far(1, BIG), 4),
        "no row": lambda: dw.group_norm_grad(_far(0, BIG), _far(0, BIG), g, 4),
        "row": lambda: dw.quantize_rows(_far(2, BIG)),
        "columns": lambda: dw.linear_i8(x, w8, g),
        "scan": lambda: dw.gated_scan(*[_far(1, 2, BIG)] * 3, g),
        "causal": lambda: dw.causal_conv(_far(1, 2, BIG), taps),
        "taps": lambda: dw.causal_conv(_far(1, 2, 8), taps),
        "map": lambda: dw.linear(x, _far(BIG, 8)),
        "map of": lambda: dw.linear(_far(2, BIG), _far(2, BIG)),
    }
    for name, call in calls.items():
        with pytest.raises(ValueError, match="2\\^31"):
            call()
            pytest.fail(name)
    for groups in (BIG, -BIG):
        with pytest.raises(ValueError, match="groups"):
            dw.group_norm(x, groups)


def test_attention_workspace_counts_rows_and_not_sequences():
    """Packed: a state for each segment that the rows are cut into, however many sequences
    they belong to, most of which are shorter than a segment."""
    heads, state = (16, 16, 128, 128), 4 * 16 * 128 * 128
    for seqs, rows in ((512, 32768), (1000, 64000), (16384, 65536), (65536, 65536)):
        for grad in (False, True):
            n = [dw.dwconv_attention_workspace_size(grad, torch.bfloat16, s, rows, True, *heads)
                 for s in (1, seqs)]
            assert n[0] == n[1]
            # a segment is at least 64 rows of 32 KB, beside which a state has 1 MB; the
            # gradient keeps two sets
            assert 0 < n[1] <= (2 if grad else 1) * state * (rows // 256), (seqs, rows, grad)
    # dense ones alike
    n = dw.dwconv_attention_workspace_size(False, torch.bfloat16, 3, 1000, False, 1, 1, 64, 64)
    assert n == 4 * 64 * 64 * (-(-3000 // 64) - 1)
