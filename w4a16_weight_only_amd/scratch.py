"""Device memory of kernels whose workgroups meet: counters that are zero before a call and zero again
after it, and scratch that needs no contents.

One block per thread and stream, kept, which the calls that a thread makes on the stream share, one after
another.  A call may be several launches with its scratch between them, and another thread's launches
may come between those, on the same stream too: so threads share none.  A thread's blocks go back to
torch's allocator when it ends.  Under capture a call has a block of the graph's own, which the
graph clears itself, so that graphs share none and need no call before.
"""
from __future__ import annotations

import threading

import torch

_KEPT_COUNTERS, _KEPT_SCRATCH = 1 << 14, 1 << 20  # bytes kept per thread and stream


class _Kept(threading.local):
    def __init__(self):
        self.blocks = {}  # by device and stream: (block, its address)


_kept = _Kept()


def _block(device, counter_bytes, scratch_bytes):
    block = torch.empty(counter_bytes + scratch_bytes, dtype=torch.uint8, device=device)
    block[:counter_bytes].zero_()
    return block


def counters_and_scratch(device: torch.device, counter_bytes: int, scratch_bytes: int) -> tuple:
    """(counters' address, scratch's address, what to hold until the call's kernels are launched), on the
    current stream of the device, which must be the current one.  For this thread alone."""
    if counter_bytes > _KEPT_COUNTERS or torch._C._cuda_isCurrentStreamCapturing():
        counter_bytes = (counter_bytes + 255) // 256 * 256
        block = _block(device, counter_bytes, scratch_bytes)
        at = block.data_ptr()
        return at, at + counter_bytes, block
    blocks = _kept.blocks
    key = (device.index, torch._C._cuda_getCurrentRawStream(device.index))
    kept = blocks.get(key)
    if kept is None:
        block = _block(device, _KEPT_COUNTERS, _KEPT_SCRATCH)
        blocks[key] = kept = (block, block.data_ptr())
    if scratch_bytes > _KEPT_SCRATCH:
        scratch = torch.empty(scratch_bytes, dtype=torch.uint8, device=device)
        return kept[1], scratch.data_ptr(), scratch
    return kept[1], kept[1] + _KEPT_COUNTERS, kept[0]
