"""Counters of kernels whose workgroups count themselves in: zero before a call, zero again after it.

One tensor per stream, kept, which calls in the stream's order share; under capture one of the
graph's own, which the graph clears itself, so that graphs share none and need no call before.
"""
from __future__ import annotations

import torch

_counters = {}  # by device and stream


def zeroed_counters(device: torch.device, nbytes: int) -> torch.Tensor:
    """Device memory of at least nbytes, zero when this stream's next kernel runs, for kernels that
    leave it zero."""
    with torch.cuda.device(device):
        if torch.cuda.is_current_stream_capturing():
            return torch.zeros(nbytes // 4, dtype=torch.int32, device=device)
        key = (device.index, torch._C._cuda_getCurrentRawStream(device.index))
        got = _counters.get(key)
        if got is None or got.numel() * 4 < nbytes:
            _counters[key] = got = torch.zeros(max(nbytes // 4, 4096), dtype=torch.int32, device=device)
        return got
