"""The Python front end of the 8-bit output head without a GPU: what it refuses before any CUDA call."""
from types import SimpleNamespace

import pytest
import torch

from canvas_sampler_gb300 import head


def test_a_stream_of_another_device_is_refused():
    """Its context would become current, and outputs and kernels would go to the wrong device."""
    ran = []
    other = SimpleNamespace(cuda_stream=1 << 20, device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream"):
        head._run(ran.append, 0, other)
    assert not ran


def _grad(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype, requires_grad=True)


CALLS = {
    "norm x": lambda: head.rmsnorm_fp8(_grad(2, 256), torch.zeros(256)),
    # (the checks of later arguments: a host tensor is refused at the first one)
    "weight": lambda: head._vector("weight", _grad(256), 256, torch.float32, 0),
    "residual": lambda: head._rows("residual", _grad(2, 256), (2, 256), (torch.float32,), 0),
    "quantise": lambda: head.quantize_fp8(_grad(2, 256)),
    "sample": lambda: head.sample_logits(_grad(2, 100), torch.zeros(2)),
}


@pytest.mark.parametrize("name", CALLS)
def test_inputs_that_want_a_gradient_are_refused(name):
    """Outputs would be cut from the graph without a word."""
    with pytest.raises(ValueError, match="gradient"):
        CALLS[name]()
    with torch.no_grad(), pytest.raises(ValueError, match="device|cuda:0"):  # (the next check)
        CALLS[name]()
