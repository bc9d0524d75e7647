"""The device and the stream of a call, for the torch front ends."""
from __future__ import annotations

import torch

# the current stream's handle without a Stream object around it, where this
# torch has the call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def check_device(dev, stream):
    """The library launches on the current device: a call whose tensors or
    stream belong to another one is refused."""
    current = torch.cuda.current_device()
    if dev.index != current:
        raise ValueError(f"tensors on {dev}, but the current device is cuda:{current}: "
                         "make theirs the current one (torch.cuda.device)")
    if stream is not None and stream.device != dev:
        raise ValueError(f"stream on {stream.device}, but the tensors are on {dev}")


def handle(stream, dev):
    """The stream's native handle, or the current one's (None: the default stream)."""
    if stream is not None:
        return stream.cuda_stream or None
    if _raw_stream is not None:
        return _raw_stream(dev.index) or None
    return torch.cuda.current_stream(dev).cuda_stream or None


def keep(stream, *tensors):
    """Orders a call on another stream than the current one, where its memory
    was allocated: that memory may have belonged to a tensor that work already
    on the current stream still uses, so the call comes after that work; and no
    memory of the call (its operands, which the caller may drop as soon as it
    returns, its results and its workspace) is handed out again before the
    other stream is done with it."""
    if stream is not None:
        current = torch.cuda.current_stream()
        if stream != current:
            stream.wait_stream(current)
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
