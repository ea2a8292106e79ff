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
