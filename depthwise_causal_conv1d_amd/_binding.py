"""What the package's binding modules share: the loaded library, the mapping of its
return codes to exceptions, and the device and stream a call runs on."""
from __future__ import annotations

# Filled in by the package, which owns the library handle.
load = None
raise_for = None
ACTIVATIONS: dict = {}


class on:
    """``with on(device index):`` that device is current inside."""

    __slots__ = ("guard",)

    def __init__(self, index):
        # most calls are for the device that is current already
        self.guard = None if index == _torch.cuda.current_device() else _torch.cuda.device(index)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


_torch = stream = None


def bind_torch(torch):
    """Called when the library is first used, so that importing the package does not
    import torch.  ``stream(index)`` is the handle of a device's current stream: without
    a stream object where this torch has that (1.7 us less a call)."""
    global _torch, stream
    _torch = torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    stream = raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)
