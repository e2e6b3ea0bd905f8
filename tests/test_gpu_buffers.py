"""The buffers that the layers keep, on streams other than the current one and under capture."""

import pytest

torch = pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402
from delayed_scaling_gemm_amd.block import NormLinearStack  # noqa: E402
from delayed_scaling_gemm_amd.linear import MXFP4Linear  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


def tokens(n, C, seed=0):
    g = torch.Generator().manual_seed(100 * seed + n)
    return torch.randn(n, C, generator=g).to(torch.bfloat16).to(DEV)


def mxfp4(C):
    torch.manual_seed(1)
    layer = MXFP4Linear(device=DEV)
    layer.quantize(torch.randn(C, C, device=DEV))
    return layer, lambda x, **kw: layer.forward(x, **kw)


def stack(C):
    torch.manual_seed(2)
    s = NormLinearStack(2, C)
    s.quantize()
    return s, lambda x, **kw: s.decode(x, **kw)


def stream_of(t):
    """Handle of the stream whose memory pool holds t."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in a segment of the allocator")


@pytest.mark.parametrize("make", [mxfp4, stack])
@pytest.mark.parametrize("as_handle", [False, True])
def test_serving_on_another_stream(make, as_handle):
    C = 256
    layer, call = make(C)
    counts = [1, 40, 7, 40, 300, 1]
    want = [call(tokens(n, C)).clone() for n in counts]
    own = set(layer._bufs)
    side = torch.cuda.Stream()
    layer, call = make(C)
    side.wait_stream(torch.cuda.current_stream())
    xs = [tokens(n, C) for n in counts]
    torch.cuda.synchronize()
    got = []
    for x in xs:
        y = call(x, stream=side.cuda_stream if as_handle else side)
        assert stream_of(y) == side.cuda_stream
        with torch.cuda.stream(side):
            got.append(y.clone())
        # memory given up by the call before must not come back on the current stream while
        # the side stream's kernels read it
        torch.empty(1 << 16, dtype=torch.uint8, device=DEV).fill_(255)
    torch.cuda.synchronize()
    assert own == set(layer._bufs)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("make", [mxfp4, stack])
@pytest.mark.parametrize("how", ["graph", "prepared"])
def test_replays_after_calls_with_other_token_counts(make, how):
    C, n = 256, 24
    layer, call = make(C)
    x = tokens(n, C)
    call(x)
    torch.cuda.synchronize()
    if how == "graph":
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = call(x)
        replay = graph.replay
    else:
        ys = []
        replay = dsg.prepare(lambda: ys.append(call(x)))
        y = ys[0]
    for k in range(3):
        call(tokens(100 + k, C))
        # what the allocator would hand out of memory that the replay still writes
        others = [torch.full(t.shape, 3, dtype=t.dtype, device=DEV) for t in layer._bufs.values()
                  for _ in range(4)]
        others += [torch.full((n, w), 3, dtype=torch.uint8, device=DEV)
                   for w in (C // 32, C // 2, C, 2 * C) for _ in range(4)]
        x.copy_(tokens(n, C, seed=k + 1))
        replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert all(bool((o == 3).all()) for o in others)
        assert torch.equal(got, call(x)), k
