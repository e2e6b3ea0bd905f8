"""Device buffers that a layer keeps from call to call.

A buffer belongs to the stream it was allocated for: the caching allocator hands freed memory on
in that stream's order.  So a layer called with ``stream=`` allocates for that stream, and the
uses of a buffer on a further stream are recorded with it: memory given up for another shape is
not handed on before the kernels queued on any of them are done.  (Which of two streams runs
first is the caller's to order, as for the layer's inputs and its state, whose fills run on the
stream that is current when the layer is made.)

A HIP graph and a prepared launch (:func:`delayed_scaling_gemm_amd.prepare`) hold addresses.  A
buffer that was used in one is kept for as long as the layer lives, also when calls with another
shape replace it; so the layer has to live as long as its graphs and prepared launches.
"""

from __future__ import annotations

import torch

from . import _recording, _stream


def _stream_object(stream, handle: int):
    if stream is None:
        return torch.cuda.current_stream()
    if not isinstance(stream, int):
        return stream
    return torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()


def _addresses_outlive_the_call() -> bool:
    return (getattr(_recording, "calls", None) is not None
            or torch.cuda.is_current_stream_capturing())


class Buffers:
    """Base of the layers: ``self.device`` and named buffers."""

    def __init__(self, device):
        self.device = torch.device(device)
        self._bufs = {}
        self._streams = {}   # name -> handles of the streams that the buffer was used on
        self._fixed = set()  # names whose buffer a graph or a prepared launch addresses
        self._replaced = []  # such buffers, after calls with other shapes

    def _held(self, name, stream=None):
        """The buffer ``name`` (or None) for a use on ``stream``."""
        t = self._bufs.get(name)
        if t is not None and self.device.type == "cuda":
            handle = _stream(stream)
            if handle not in self._streams[name]:
                t.record_stream(_stream_object(stream, handle))
                self._streams[name].add(handle)
            if _addresses_outlive_the_call():
                self._fixed.add(name)
        return t

    def _buf(self, name, shape, dtype, stream=None):
        """The buffer ``name`` for a use on ``stream``, a new one where shape or type changed."""
        t = self._bufs.get(name)
        if t is not None and t.shape == shape and t.dtype == dtype:
            return self._held(name, stream)
        if self.device.type != "cuda":
            t = torch.empty(shape, dtype=dtype, device=self.device)
        else:
            handle = _stream(stream)
            with torch.cuda.stream(_stream_object(stream, handle)):
                t = torch.empty(shape, dtype=dtype, device=self.device)
            self._streams[name] = {handle}
            if name in self._fixed:
                self._replaced.append(self._bufs[name])
                self._fixed.discard(name)
            if _addresses_outlive_the_call():
                self._fixed.add(name)
        self._bufs[name] = t
        return t
