"""Which workspace a call that brings none gets: whose memory, and with whom it
is shared.  Torch's streams are replaced by a model of them (no GPU)."""
import contextlib
import threading

import pytest
import torch

from online_activation_aware_ttq_amd import _binding

CPU = torch.device("cpu")


class Streams:
    """The current stream, the ones under capture, and on which stream each
    buffer was taken."""

    def __init__(self, monkeypatch):
        self.now, self.capturing, self.taken = 5, set(), {}
        monkeypatch.setattr(_binding, "_current_stream", lambda dev: self.now)
        monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing",
                            lambda: self.now in self.capturing, raising=False)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
        monkeypatch.setattr(torch.cuda, "stream", self.on)

    @contextlib.contextmanager
    def on(self, handle):
        before, self.now = self.now, handle
        yield
        self.now = before


@pytest.fixture
def streams(monkeypatch):
    _binding._host()
    s = Streams(monkeypatch)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda *a: None)
    monkeypatch.setattr(_binding, "_SCRATCH", type(_binding._SCRATCH)())
    empty = torch.empty

    def record(*a, **kw):
        t = empty(*a, **kw)
        s.taken[t.data_ptr()] = s.now
        return t

    monkeypatch.setattr(torch, "empty", record)
    return s


def get(stream, need, step):
    if step:
        return _binding._step_workspace(CPU, stream, need, None)
    return _binding._workspace(CPU, stream, None, lambda: need)


STEP = pytest.mark.parametrize("step", [False, True], ids=["projection", "step"])


@STEP
def test_kept_between_a_threads_calls_on_a_stream(streams, step):
    a = get(5, 1000, step)
    assert get(5, 900, step) is a and a.numel() >= 1000
    b = get(5, 5000, step)
    assert b.numel() >= 5000 and get(5, 1000, step) is b
    assert get(6, 1000, step) is not b


@STEP
def test_two_threads_on_one_stream_share_none(streams, step):
    mine, theirs = get(5, 1000, step), []
    t = threading.Thread(target=lambda: theirs.append(get(5, 1000, step)))
    t.start()
    t.join()
    assert theirs[0].data_ptr() != mine.data_ptr()
    assert get(5, 1000, step) is mine


@STEP
def test_a_captured_call_has_its_own(streams, step):
    kept = get(5, 1000, step)
    streams.capturing.add(5)
    a, b = get(5, 1000, step), get(5, 1000, step)
    streams.capturing.clear()
    assert len({t.data_ptr() for t in (kept, a, b)}) == 3
    assert get(5, 1000, step) is kept


@STEP
def test_a_capture_on_a_stream_given_as_argument(streams, step):
    """Stream 9 is captured, torch's current one is not, and the other way round."""
    kept = get(9, 1000, step)
    streams.capturing.add(9)
    a, b = get(9, 1000, step), get(9, 1000, step)
    assert len({t.data_ptr() for t in (kept, a, b)}) == 3
    assert get(9, 1000, step) is not kept
    streams.capturing.clear()
    streams.capturing.add(5)
    assert get(9, 1000, step) is kept


@STEP
def test_memory_is_taken_on_the_stream_that_uses_it(streams, step):
    for stream in (5, 11):
        assert streams.taken[get(stream, 3000, step).data_ptr()] == stream
    assert streams.now == 5
