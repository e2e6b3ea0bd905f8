"""Device buffers that a layer keeps from call to call.

A buffer belongs to the stream it was allocated for: the caching allocator hands freed memory on
in that stream's order.  So a layer called with ``stream=`` allocates for that stream, and when
it is called on a further one, that use of its buffers is recorded with them: memory given up for
another shape is not handed on before the kernels queued on any of them are done.  (Which of two
streams runs first is the caller's to order, as for the layer's inputs and its state, whose fills
run on the stream that is current when the layer is made.)

A HIP graph and a prepared launch (:func:`delayed_scaling_gemm_amd.prepare`) hold addresses.  The
buffers that a layer has while one is made are kept for as long as the layer lives, also when calls
with another shape replace them; so the layer has to live as long as its graphs and prepared
launches.

Both are looked at once per call, not per buffer: a step of 15 buffers took 18 us more on the host
(43, then 61) when each of them asked for the stream and for a capture.
"""

from __future__ import annotations

import torch

from . import _current_stream, _recording, _stream


class Buffers:
    """Base of the layers: ``self.device`` and named buffers."""

    def __init__(self, device):
        self.device = torch.device(device)
        self._bufs = {}
        self._handle = None     # of the stream of the last call
        self._seen = {}         # name -> handles of the streams that the buffer was used on
        self._outlive = False   # a graph or a prepared launch is being made
        self._fixed = set()     # names of the buffers that one may address
        self._replaced = []     # such buffers, after calls with other shapes

    def _use(self, stream):
        """Start of a call that works on ``stream`` (a stream, its handle, or None: the current
        one)."""
        if self.device.type != "cuda":
            return
        handle = _stream(stream)
        if handle != self._handle:
            self._handle = handle
            for name, t in self._bufs.items():
                if handle not in self._seen[name]:
                    t.record_stream(self._stream_object())
                    self._seen[name].add(handle)
        self._outlive = (getattr(_recording, "calls", None) is not None
                         or torch.cuda.is_current_stream_capturing())
        if self._outlive:
            self._fixed.update(self._bufs)

    def _stream_object(self):
        if self._handle == _current_stream():
            return torch.cuda.current_stream()
        return (torch.cuda.ExternalStream(self._handle) if self._handle
                else torch.cuda.default_stream())

    def _buf(self, name, shape, dtype):
        """The buffer ``name``, a new one where shape or type changed."""
        t = self._bufs.get(name)
        if t is not None and t.shape == shape and t.dtype == dtype:
            return t
        if self.device.type != "cuda":
            t = torch.empty(shape, dtype=dtype, device=self.device)
        else:
            if self._handle is None:
                self._use(None)
            with torch.cuda.stream(self._stream_object()):
                t = torch.empty(shape, dtype=dtype, device=self.device)
            if name in self._fixed:
                self._replaced.append(self._bufs[name])
                self._fixed.discard(name)
            if self._outlive:
                self._fixed.add(name)
            self._seen[name] = {self._handle}
        self._bufs[name] = t
        return t
