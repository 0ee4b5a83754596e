"""What every call of the binding needs: the stream, the device, the checks."""
from __future__ import annotations

import torch


def _stream_ptr(stream, device) -> int:
    s = torch.cuda.current_stream(device) if stream is None else stream
    return s.cuda_stream


def _on_device(dev: torch.device, fn, *args) -> int:
    """Call fn with dev as the current CUDA device (switching only if needed)."""
    if dev.index is None or dev.index == torch.cuda.current_device():
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _req(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)
