"""Kept scratch (scratch.py) on the CPU: which calls share a block.  The current stream is set from here, and
the blocks are host memory."""
from __future__ import annotations

import threading

import pytest
import torch

from w4a16_weight_only_amd import _lib
from w4a16_weight_only_amd.scratch import counters_and_scratch

CPU = torch.device("cpu")
# What the two operators ask for: a layer's counters and workspace, a fused product's splits.
LAYER, FUSED = (_lib.AWQ_MOE_LAYER_COUNTERS, 600_000), (64, 131072)


@pytest.fixture
def stream(monkeypatch):
    now = {"raw": 0, "capturing": False}
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: now["capturing"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: now["raw"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentStream", lambda device: (now.get("id", 0), 0, 1), raising=False)
    return now


def ranges(got, sizes):
    """The byte ranges of a call's counters and scratch."""
    return [(at, at + n) for at, n in zip(got[:2], sizes)]


def apart(a, b):
    return all(p[1] <= q[0] or q[1] <= p[0] for p in a for q in b)


def in_thread(f):
    got, done = [], threading.Event()
    stay = threading.Event()

    def run():
        got.append(f())
        done.set()
        stay.wait(30)

    t = threading.Thread(target=run)
    t.start()
    assert done.wait(30)
    return got[0], lambda: (stay.set(), t.join())


@pytest.mark.parametrize("here,there", [(LAYER, FUSED), (FUSED, LAYER), (LAYER, LAYER), (FUSED, FUSED)],
                         ids=["layer-fused", "fused-layer", "layer-layer", "fused-fused"])
def test_two_threads_on_one_stream_share_nothing(stream, here, there):
    """A call of one thread may be enqueued between the launches of another's: a layer's second launch would find
    a fused product's sums in the place of its tickets and counts."""
    first = counters_and_scratch(CPU, *here)
    other, end = in_thread(lambda: counters_and_scratch(CPU, *there))
    try:
        assert apart(ranges(first, here), ranges(other, there))
    finally:
        end()


def test_a_thread_keeps_its_block_for_a_stream(stream):
    a, b = counters_and_scratch(CPU, *LAYER), counters_and_scratch(CPU, *FUSED)
    assert a[:2] == b[:2]
    assert apart(ranges(a, LAYER)[:1], ranges(a, LAYER)[1:])
    stream["raw"] = 4096
    assert apart(ranges(a, LAYER), ranges(counters_and_scratch(CPU, *LAYER), LAYER))
    stream["raw"] = 0
    assert counters_and_scratch(CPU, *LAYER)[:2] == a[:2]
    large = (64, 8 << 20)
    assert apart(ranges(a, LAYER), ranges(counters_and_scratch(CPU, *large), large)[1:])


def test_captured_calls_have_their_own(stream):
    a = counters_and_scratch(CPU, *LAYER)
    stream["capturing"] = True
    b, c = (counters_and_scratch(CPU, *FUSED) for _ in range(2))
    assert apart(ranges(a, LAYER), ranges(b, FUSED)) and apart(ranges(b, FUSED), ranges(c, FUSED))
    for got in (b, c):
        assert not got[2][:FUSED[0]].any()  # zero counters


def test_blocks_go_with_their_thread(stream):
    """What a thread kept is not held by anyone after it."""
    import weakref

    def run():
        return weakref.ref(counters_and_scratch(CPU, *LAYER)[2])

    alive, end = in_thread(run)
    assert alive() is not None
    end()
    assert alive() is None


def test_streams_from_outside_keep_nothing(stream):
    """Their handles come back for other streams, in no order with what ran before: torch gives such a stream its
    handle for an id, its own streams small ones."""
    stream.update(raw=1 << 40, id=1 << 40)
    first = counters_and_scratch(CPU, *LAYER)
    second = counters_and_scratch(CPU, *LAYER)
    assert apart(ranges(first, LAYER), ranges(second, LAYER)) and not second[2][:LAYER[0]].any()
    stream.update(raw=1 << 41, id=35)
    assert counters_and_scratch(CPU, *LAYER)[:2] == counters_and_scratch(CPU, *LAYER)[:2]
    stream.update(raw=0, id=0)  # the default stream
    assert counters_and_scratch(CPU, *LAYER)[:2] == counters_and_scratch(CPU, *LAYER)[:2]
