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

    __slots__ = ("dev", "guard")

    def __init__(self, dev):
        self.dev = dev

    def __enter__(self):
        import torch

        self.guard = None
        if self.dev.index is not None and self.dev.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(self.dev)
            self.guard.__enter__()
        return torch.cuda.current_stream(self.dev).cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)
