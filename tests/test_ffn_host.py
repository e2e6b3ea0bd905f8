"""GatedFeedForwardStack's checks of its arguments and of the order of its calls (no GPU: the library
calls are stand-ins)."""

import pytest
import torch

from delayed_scaling_gemm_amd import ffn

X = torch.zeros(4, 64, dtype=torch.bfloat16)


@pytest.fixture
def stack(monkeypatch):
    for name in dir(ffn):
        if name.startswith("fp8ds_"):
            monkeypatch.setattr(ffn, name, lambda *a, **k: 256)
    return ffn.GatedFeedForwardStack(2, 64, 160, device="cpu")


@pytest.mark.parametrize("layers,width,inner", [(0, 64, 64), (2, 0, 64), (2, 40, 64), (1, 64, 100), (1, 64, 0)])
def test_shapes_refused(layers, width, inner):
    with pytest.raises(ValueError):
        ffn.GatedFeedForwardStack(layers, width, inner, device="cpu")


def test_stream_type_refused():
    with pytest.raises(TypeError):
        ffn.GatedFeedForwardStack(1, 64, 64, stream_dtype=torch.float16, device="cpu")


def test_order_of_calls(stack):
    with pytest.raises(RuntimeError):
        stack.backward(X)
    with pytest.raises(RuntimeError):
        stack.optimizer_step(1e-3, 1.0)
    with pytest.raises(RuntimeError):
        stack.decode(X)
    for _ in range(2):
        stack.forward(X), stack.backward(X), stack.optimizer_step(1e-3, 1.0)
        with pytest.raises(RuntimeError, match="once after each"):
            stack.optimizer_step(1e-3, 1.0)
    stack.forward(X)
    with pytest.raises(RuntimeError, match="backward"):
        stack.optimizer_step(1e-3, 1.0)
    with pytest.raises(RuntimeError, match="pending"):
        stack.quantize()
    stack.backward(X), stack.quantize(), stack.decode(X)
    for bad in (torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)):
        for call in (stack.forward, stack.decode):
            with pytest.raises(ValueError):
                call(bad)
    stack.forward(X)
    with pytest.raises(RuntimeError, match="this shape"):
        stack.backward(torch.zeros(3, 64, dtype=torch.bfloat16))


def test_gradients_match_parameters(stack):
    stack.forward(X), stack.backward(X)
    shapes = [tuple(g.shape) for g in stack.grads()]
    assert shapes == [tuple(p.shape) for p in stack.w + stack.wd + stack.vectors()]
