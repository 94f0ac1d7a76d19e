"""The sequence operators' largest batches, without a GPU: row and sequence
counts whose 32-bit arithmetic the kernels could not carry are refused.  Fake
device addresses; every call returns before any launch."""
import os
import re

import pytest

import depthwise_convolution_amd as dw

A = 1 << 40
X, W, Y, Z, P, Q, R, S, U, V = (A + (k << 36) for k in range(10))     # 64 GiB apart
TOP = dw.SEQ_MAX_ROWS
# beyond the most rows, dense and packed: the last one that 32 bits hold, and one more
# than allowed; and more sequences than that
BATCHES = [(1, (1 << 31) - 1, None), (1, TOP + 1, None), (2, TOP // 2 + 1, None),
           (5, TOP + 1, V), (5, (1 << 31) - 1, V), (TOP + 1, 0, V), ((1 << 31) - 1, 1, None)]


def test_header_agrees():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                        "dwconv_seq.h")
    assert int(re.search(r"DWCONV_SEQ_MAX_ROWS\s+(\d+)", open(path).read()).group(1)) == TOP


def _status(name, *args):
    return dw.STATUS[getattr(dw.lib(), name)(*args)]


@pytest.mark.parametrize("seqs,tokens,offsets", BATCHES)
def test_batches_past_the_limit(seqs, tokens, offsets):
    import ctypes
    batch, big, packed = (seqs, tokens, offsets), 1 << 50, int(offsets is not None)
    assert _status("dwconv_causal_fwd", X, 1, 1, W, 0, None, 0, None, Y, 1, None, *batch, 1, 2,
                   None) == "BAD_DIM"
    assert _status("dwconv_causal_grad", Y, 1, X, 1, 1, W, 0, None, 0, None, None, Z, 1, P, None,
                   None, U, big, *batch, 1, 2, None) == "BAD_DIM"
    assert _status("dwconv_scan_fwd", X, 1, P, 1, Q, 1, 1, W, 8.0, None, Y, 1, None, None, U, big,
                   *batch, 1, None) == "BAD_DIM"
    assert _status("dwconv_scan_grad", Y, 1, X, 1, P, 1, Q, 1, 1, W, 8.0, S, None, Z, 1, R, 1,
                   R + (1 << 35), 1, W + 64, None, U, big, *batch, 1, None) == "BAD_DIM"
    n = ctypes.c_longlong(0)
    for name, tail in (("dwconv_scan_states_size", (1,)), ("dwconv_causal_grad_workspace_size",
                                                           (1, 2))):
        assert _status(name, seqs, tokens, packed, *tail, ctypes.byref(n)) == "BAD_DIM"
    assert _status("dwconv_scan_workspace_size", 0, seqs, tokens, packed, 1,
                   ctypes.byref(n)) == "BAD_DIM"


@pytest.mark.parametrize("rows", [TOP + 1, (1 << 31) - 1])
def test_rows_past_the_limit(rows):
    assert _status("dwconv_causal_step", X, 1, 1, W, 0, None, 0, Z, Y, 1, rows, 1, 2,
                   None) == "BAD_DIM"
    assert _status("dwconv_scan_step", X, 1, P, 1, Q, 1, 1, W, 8.0, Z, Y, 1, rows, 1,
                   None) == "BAD_DIM"
    assert _status("dwconv_linear_fwd", X, 1, W, 1, 1, None, 0, None, 0, Y, 1, None, 0, U, 1 << 50,
                   rows, 1, 1, None) == "BAD_DIM"
    assert _status("dwconv_linear_grad", Y, 1, X, 1, W, 1, 1, 0, None, 0, Z, 1, P, 1, Q, U,
                   1 << 50, rows, 1, 1, None) == "BAD_DIM"
    assert _status("dwconv_linear_describe", 0, 1, 1, rows, 1, 1, None, 0, None) == "BAD_DIM"
