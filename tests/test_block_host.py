"""NormLinearStack's checks of its arguments and of the order of its calls (no GPU)."""

import pytest
import torch

from delayed_scaling_gemm_amd.block import NormLinearStack


@pytest.mark.parametrize("layers,width", [(0, 64), (2, 0), (2, 48), (1, -32)])
def test_shapes_refused(layers, width):
    with pytest.raises(ValueError):
        NormLinearStack(layers, width, device="cpu")


def test_stream_type_refused():
    with pytest.raises(TypeError):
        NormLinearStack(1, 64, stream_dtype=torch.float16, device="cpu")


def test_order_and_shapes_of_calls():
    s = NormLinearStack(2, 64, device="cpu")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(RuntimeError):
        s.backward(x)
    with pytest.raises(RuntimeError):
        s.optimizer_step(1e-3, 1.0)
    with pytest.raises(RuntimeError):
        s.decode(x)
    for bad in (torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            s.forward(bad)
