"""The binding's own scratch of the calls over a part of the cache, on the host
(streams and captures stood in for): streams that may run beside one another
and captures never share a buffer."""

import weakref

import pytest
import torch

import paged_gqa_decode_reshape_gb300 as pg

DEV = torch.device("cpu", 0)


class Streams:
    """What the binding asks about the current stream."""

    def __init__(self, mp):
        self.handle, self.capture = 0, 0
        mp.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: self.handle)
        mp.setattr(torch._C, "_cuda_getDevice", lambda: 0)
        mp.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: self.capture != 0)
        mp.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.capture != 0)
        mp.setattr(pg, "pa_capture_id", lambda stream: self.capture, raising=False)

        def call(*a):  # an entry point: its workspace and stream come last
            self.seen = a[-3:]
            return 0

        mp.setattr(pg, "_lookup", lambda key: (call, self.need))

    def __call__(self, need, handle=0, capture=0):
        """(address, bytes) of the workspace that a call on this stream is given."""
        self.need, self.handle, self.capture = need, handle, capture
        pg._run("pa_decode_window", DEV, (), None, (1, 1, 1, 64))
        assert self.seen[2] == handle
        return self.seen[:2]


@pytest.fixture
def on(monkeypatch):
    monkeypatch.setattr(pg, "_subset_ws", pg._Scratch())
    monkeypatch.setattr(pg, "_calls", {})
    return Streams(monkeypatch)


def apart(a, b):
    return a[0] + a[1] <= b[0] or b[0] + b[1] <= a[0]


def test_streams_have_buffers_of_their_own(on):
    a, b = on(1000, handle=0), on(1000, handle=7)
    assert a[1] >= 1000 and b[1] >= 1000 and apart(a, b)
    assert on(1000, handle=0) == a and on(500, handle=7) == b  # kept per stream
    c = on(90_000, handle=7)
    assert c[1] >= 90_000 and on(1000, handle=0) == a


def test_captures_have_buffers_of_their_own(on):
    a = on(1000, handle=3)
    b = on(1000, handle=3, capture=11)  # captured on the stream of the eager call
    assert apart(a, b)
    assert on(800, handle=3, capture=11) == b  # one buffer for the calls of a capture
    fork = on(1000, handle=4, capture=11)  # a second stream in the same capture
    assert apart(fork, b) and apart(fork, a)
    held = pg._subset_ws.get(DEV, 1000, 3)
    assert held.data_ptr() == b[0]
    c = on(1000, handle=3, capture=12)
    assert apart(c, b) and apart(c, a)
    assert on(1000, handle=3) == a


def test_a_capture_before_any_call_is_refused(on):
    with pytest.raises(RuntimeError, match="before the capture"):
        on(1000, handle=3, capture=11)
    on(1000, handle=0)
    on(1000, handle=3, capture=11)
    with pytest.raises(RuntimeError, match="before the capture"):
        on(5000, handle=3, capture=11)


def test_captures_in_turn_keep_their_buffers(on):
    """Captures of several threads, whose calls come in turn."""
    on(1000, handle=0)
    held = []
    for _ in range(3):
        for handle, capture in ((3, 11), (4, 12)):
            on(1000, handle=handle, capture=capture)
            held.append(pg._subset_ws.held(0, handle))
    assert all(h is held[i % 2] for i, h in enumerate(held)) and held[0] is not held[1]


@pytest.mark.parametrize("pooled", [False, True])
def test_buffers_outside_a_graphs_pool_are_kept(on, monkeypatch, pooled):
    """A graph that was not captured into a memory pool of its own holds its buffer's address for good."""
    monkeypatch.setattr(pg, "_in_graph_pool", lambda buf: pooled)
    on(1000, handle=0)
    on(1000, handle=3, capture=100)
    first = weakref.ref(pg._subset_ws.held(0, 3))
    for i in range(20):
        on(1000, handle=3, capture=200 + i)
    assert (first() is None) == pooled
