"""The binding's checks of devices, on stand-ins for a second GPU: a workspace or
a stream of another device than the tensors' is refused before anything is
enqueued there."""
import types

import pytest
import torch

import depthwise_convolution_amd as dw
from depthwise_convolution_amd import sequence


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on GPU `index`."""
    index = 0
    is_cuda = True

    def get_device(self):
        return self.index

    @property
    def device(self):
        return torch.device("cuda", self.index)


class OnOther(OnGpu):
    index = 1


def _tensor(kind, *shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(kind)


def test_workspace_of_another_device():
    x = _tensor(OnGpu, 4, 8)
    sequence._setup()
    here = _tensor(OnGpu, 64, dtype=torch.uint8)
    assert sequence._space(here, x) == (here.data_ptr(), 64)
    assert sequence._space(None, x) == (None, 0)
    for other in (_tensor(OnOther, 64, dtype=torch.uint8), torch.zeros(64, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="workspace must be on the GPU device of x"):
            sequence._space(other, x)
    with pytest.raises(TypeError, match="workspace"):
        sequence._space(4096, x)
    with pytest.raises(ValueError, match="contiguous"):
        sequence._space(_tensor(OnGpu, 8, 8, dtype=torch.uint8)[:, :4], x)


def test_stream_of_another_device():
    x = _tensor(OnGpu, 2, 3, 8)
    other = types.SimpleNamespace(cuda_stream=5, device=torch.device("cuda", 1))
    calls = [lambda: dw.causal_conv(x, x[0], stream=other),
             lambda: dw.causal_conv_step(x[0], x, x[0], stream=other),
             lambda: dw.gated_scan(x, x, x, x[0, 0], stream=other),
             lambda: dw.gated_scan_step(x[0], x[0], x[0], x[0, 0], x[0], stream=other),
             lambda: dw.linear(x, x[0], stream=other),
             lambda: dw.linear_grad(x, x, x[0], stream=other)]
    for call in calls:
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call()
