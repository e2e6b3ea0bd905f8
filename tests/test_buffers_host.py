"""The buffers that the layers keep from call to call, and streams (no GPU: the library calls and
torch's stream calls are stand-ins, only the host's bookkeeping runs)."""

import contextlib
import gc
import weakref

import pytest
import torch

import delayed_scaling_gemm_amd as dsg
from delayed_scaling_gemm_amd import block, linear

BF = torch.bfloat16


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


class World:
    """What was allocated while which stream was current, and which uses were recorded."""

    def __init__(self):
        self.current, self.allocated, self.recorded = 0, {}, []


@pytest.fixture
def world(monkeypatch):
    w = World()
    empty = torch.empty

    def fake_empty(*a, device=None, **kw):
        t = empty(*a, **kw)
        w.allocated[t.data_ptr()] = w.current
        return t

    @contextlib.contextmanager
    def on(s):
        before, w.current = w.current, s.cuda_stream
        yield
        w.current = before

    for mod in (linear, block):
        for name in dir(mod):
            if name.startswith("fp8ds_") and not name.endswith("workspace"):
                monkeypatch.setattr(mod, name, lambda *a, **k: None)
    monkeypatch.setattr(torch, "empty", fake_empty)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: FakeStream(w.current))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: FakeStream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, *a: FakeStream(h))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(dsg, "_raw_stream", lambda: w.current)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: w.recorded.append((t.data_ptr(), s.cuda_stream)), raising=False)
    return w


def layers():
    """Each layer with a call of it for a number of tokens."""
    C = 64
    x = lambda m: torch.zeros(m, C, dtype=BF)  # noqa: E731
    w = torch.zeros(C, C)
    mx4 = linear.MXFP4Linear(device="cpu")
    yield mx4, lambda m, s: (mx4.quantize(w, s), mx4.forward(x(m), stream=s))
    mx4s = linear.MXFP4Linear(device="cpu")
    yield mx4s, lambda m, s: mx4s.step(x(m), w, x(m), stream=s)
    mx8 = linear.MXLinear(device="cpu")
    yield mx8, lambda m, s: mx8.step(x(m), w, x(m), stream=s)
    lin = linear.DelayedScalingLinear(device="cpu")
    yield lin, lambda m, s: (lin.step(x(m), w, x(m), stream=s),
                             lin.adamw_step(w, w, w, 1e-3, 1, stream=s))
    batch = linear.BatchedDelayedScalingLinear(2, device="cpu")
    yield batch, lambda m, s: batch.step(torch.zeros(2, m, C, dtype=BF),
                                         torch.zeros(2, C, C, dtype=BF), stream=s)
    st = block.NormLinearStack(2, C, device="cpu")

    def train(m, s):
        st.forward(x(m), s), st.backward(x(m), s), st.optimizer_step(1e-3, 1.0, stream=s)

    yield st, train
    sv = block.NormLinearStack(2, C, device="cpu")
    yield sv, lambda m, s: (sv.quantize(s), sv.decode(x(m), stream=s))


@pytest.fixture(params=range(7), ids=["mxfp4-forward", "mxfp4-step", "mx-step", "linear", "batched",
                                      "stack-train", "stack-decode"])
def layer(request, world, monkeypatch):
    import delayed_scaling_gemm_amd as pkg

    for name in ("fp8ds_cast_batched", "fp8ds_gemm_batched", "fp8ds_linear_batched"):
        monkeypatch.setattr(pkg, name, lambda *a, **k: None)
    monkeypatch.setattr(block, "fp8ds_rmsnorm_bwd_workspace", lambda *a: 256)
    monkeypatch.setattr(block, "fp8ds_grad_norm_workspace", lambda *a: 256)
    obj, call = list(layers())[request.param]
    obj.device = torch.device("cuda")  # (allocations are on the host all the same)
    return obj, call


@pytest.mark.parametrize("stream", [FakeStream(7), 7])
def test_buffers_belong_to_the_stream_that_uses_them(layer, world, stream):
    obj, call = layer
    for tokens in (32, 96):  # the second call's buffers take the place of the first's
        call(tokens, stream)
        assert {world.allocated[t.data_ptr()] for t in obj._bufs.values()} == {7}
    assert not world.recorded


def test_use_on_a_further_stream_is_recorded(layer, world):
    obj, call = layer
    call(32, None)
    assert {world.allocated[t.data_ptr()] for t in obj._bufs.values()} == {0}
    kept = {t.data_ptr() for t in obj._bufs.values()}
    call(32, FakeStream(9))
    assert {t.data_ptr() for t in obj._bufs.values()} == kept
    assert {p for p, s in world.recorded if s == 9} == kept
    n = len(world.recorded)
    call(32, FakeStream(9)), call(32, None)
    assert len(world.recorded) == n  # once for each stream


@pytest.mark.parametrize("how", ["captured", "prepared"])
def test_buffers_of_captured_and_prepared_launches_stay(layer, world, monkeypatch, how):
    """A graph and a prepared launch hold addresses: another shape must not free them."""
    obj, call = layer
    call(32, None)
    if how == "captured":
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
        call(32, None)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    else:
        launch = dsg.prepare(lambda: call(32, None))
        assert callable(launch)
    held = [weakref.ref(t) for t in obj._bufs.values()]
    call(96, None), call(64, None)
    gc.collect()
    assert all(r() is not None for r in held)
    # and what no graph knows is given up
    eager = {n: (weakref.ref(t), t.shape) for n, t in obj._bufs.items()}
    call(128, None)
    gc.collect()
    changed = [r for n, (r, shape) in eager.items() if obj._bufs[n].shape != shape]
    assert changed and all(r() is None for r in changed)
