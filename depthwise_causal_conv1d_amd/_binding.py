"""What the package's binding modules share: the loaded library, the mapping of its
return codes to exceptions, and the device and stream a call runs on."""
from __future__ import annotations

# Filled in by the package, which owns the library handle.
load = None
raise_for = None
ACTIVATIONS: dict = {}


class on:
    """``with on(device) as stream``: the device is current inside, ``stream`` its
    current stream's handle."""

    __slots__ = ("index", "guard")

    def __init__(self, dev):
        self.index = dev.index

    def __enter__(self):
        current = _torch.cuda.current_device()
        index = current if self.index is None else self.index
        self.guard = None
        if index != current:
            self.guard = _torch.cuda.device(index)
            self.guard.__enter__()
        return _stream(index)

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _raw_stream():
    """The handle of a device's current stream: without a stream object where this torch
    has that (1.7 us less a call)."""
    raw = getattr(_torch._C, "_cuda_getCurrentRawStream", None)
    return raw or (lambda index: _torch.cuda.current_stream(index).cuda_stream)


_torch = _stream = None


def bind_torch(torch):
    """Called when the library is loaded, so that importing the package does not import torch."""
    global _torch, _stream
    _torch = torch
    _stream = _raw_stream()
