"""What every call of the binding needs: the stream, the device, the checks."""
from __future__ import annotations

import torch


# The current stream's handle, without a Stream object around it (0.1 against 2 us
# on the host, of some 10 a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


# CUDA is initialised by then: the calls' tensors are on the device.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_ptr(stream, device) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _on_device(dev: torch.device, fn, *args) -> int:
    """Call fn with dev as the current CUDA device (switching only if needed)."""
    if dev.index is None or dev.index == _current_device():
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _req(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)
