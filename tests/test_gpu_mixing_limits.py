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
