"""Device memory of kernels whose workgroups meet: counters that are zero before a call and zero again
after it, and scratch that needs no contents.

One block per thread and stream, kept, which the calls that a thread makes on the stream share, one after
another.  A call may be several launches with its scratch between them, and another thread's launches
may come between those, on the same stream too: so threads share none.  A thread's blocks go back to
torch's allocator when it ends.  Kept are those of torch's own streams, which last as long as the
process and are few; a stream from outside may be destroyed with work under way and its handle given
to the next, so a call there has a block of its own (a fill and an allocation more).  Under capture a call has
a block of the graph's own, which the graph clears itself, so that graphs share none and need no call
before.
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


def _of_one_call(device, counter_bytes, scratch_bytes):
    counter_bytes = (counter_bytes + 255) // 256 * 256
    block = _block(device, counter_bytes, scratch_bytes)
    at = block.data_ptr()
    return at, at + counter_bytes, block


def counters_and_scratch(device: torch.device, counter_bytes: int, scratch_bytes: int) -> tuple:
    """(counters' address, scratch's address, what to hold until the call's kernels are launched), on the
    current stream of the device, which must be the current one.  For this thread alone."""
    if counter_bytes > _KEPT_COUNTERS or torch._C._cuda_isCurrentStreamCapturing():
        return _of_one_call(device, counter_bytes, scratch_bytes)
    blocks = _kept.blocks
    stream = torch._C._cuda_getCurrentRawStream(device.index)
    key = (device.index, stream)
    kept = blocks.get(key)
    if kept is None:
        if stream != 0 and torch._C._cuda_getCurrentStream(device.index)[0] == stream:
            return _of_one_call(device, counter_bytes, scratch_bytes)  # a stream from outside: its id is its handle
        block = _block(device, _KEPT_COUNTERS, _KEPT_SCRATCH)
        blocks[key] = kept = (block, block.data_ptr())
    if scratch_bytes > _KEPT_SCRATCH:
        scratch = torch.empty(scratch_bytes, dtype=torch.uint8, device=device)
        return kept[1], scratch.data_ptr(), scratch
    return kept[1], kept[1] + _KEPT_COUNTERS, kept[0]
