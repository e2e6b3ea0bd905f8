"""NormLinearStack's order of calls (no GPU: the library calls are stand-ins)."""

import pytest
import torch

from delayed_scaling_gemm_amd import block

X = torch.zeros(4, 64, dtype=torch.bfloat16)


@pytest.fixture
def stack(monkeypatch):
    for name in dir(block):
        if name.startswith("fp8ds_"):
            monkeypatch.setattr(block, name, lambda *a, **k: 256)
    return block.NormLinearStack(2, 64, device="cpu")


def step(s):
    s.forward(X), s.backward(X), s.optimizer_step(1e-3, 1.0)


def test_one_optimizer_step_for_a_backward(stack):
    step(stack)
    with pytest.raises(RuntimeError, match="backward"):
        stack.optimizer_step(1e-3, 1.0)
    step(stack)


def test_no_optimizer_step_between_forward_and_backward(stack):
    """It would write the FP8 weights that the pending backward() reads."""
    step(stack)
    stack.forward(X), stack.backward(X)
    stack.forward(X)
    with pytest.raises(RuntimeError, match="backward"):
        stack.optimizer_step(1e-3, 1.0)
    stack.backward(X)  # its own forward's weights are untouched
    stack.optimizer_step(1e-3, 1.0)


def test_forwards_without_a_backward_and_skipped_steps(stack):
    stack.forward(X), stack.forward(X), stack.backward(X)
    stack.forward(X), stack.backward(X)  # a step left out
    stack.optimizer_step(1e-3, 1.0)
