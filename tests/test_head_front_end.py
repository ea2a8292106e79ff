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


BAD_NAMES = {
    "fp8": lambda: head._choice("fp8", head._FP8, "e4m3fn"),
    "out_dtype": lambda: head._choice("out_dtype", head._OUT, torch.bfloat16),
    "impl": lambda: head._choice("impl", head._IMPLS, "fast"),
    "unhashable": lambda: head._choice("impl", head._IMPLS, ["simt"]),
}


@pytest.mark.parametrize("name", BAD_NAMES)
def test_unknown_names_are_refused_with_the_known_ones(name):
    with pytest.raises(ValueError, match="must be one of"):
        BAD_NAMES[name]()


def test_the_functions_that_take_names_look_them_up_so():
    import inspect
    for f, n in ((head.rmsnorm_fp8, 1), (head.quantize_fp8, 1), (head.matmul_fp8, 2), (head.OutputHead, 2)):
        assert inspect.getsource(f).count("_choice(") == n, f


def test_numbers_that_do_not_fit_are_refused():
    """Not as an error of the packing: 2^31 columns, an eps that no float holds."""
    from canvas_sampler_gb300 import _lib as C
    if not C.os.path.exists(C.LIB_PATH):
        from canvas_sampler_gb300 import build
        build.build()
    zeros = [0] * 10
    with pytest.raises(ValueError, match="ds_quantize_fp8"):
        head._call("ds_quantize_fp8", 0, 1, 1 << 31, *zeros[:9])
    with pytest.raises(ValueError, match="ds_rmsnorm_fp8"):
        head._call("ds_rmsnorm_fp8", 0, 1, 128, 0, 0, 1e300, 0.0, 0, *zeros)


def test_without_pytorchs_private_helpers():
    """Where a PyTorch lacks the cheap forms, the public ones serve."""
    import subprocess
    import sys
    code = ("import torch\n"
            "for m, n in ((torch._C, '_cuda_getDevice'), (torch._C, '_cuda_getCurrentRawStream'),\n"
            "             (torch._C._dynamo.guards, '_empty_strided_cuda')):\n"
            "    if hasattr(m, n): delattr(m, n)\n"
            "from canvas_sampler_gb300 import head\n"
            "assert head._current_device is torch.cuda.current_device\n"
            "assert callable(head._raw_stream) and callable(head._empty_strided_cuda)\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
