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


class Fake:
    """What the entry points ask of a GPU tensor."""

    def __init__(self, shape, dtype):
        self.shape = torch.Size([shape] if isinstance(shape, int) else shape)
        self.dtype, self.device = dtype, torch.device("cuda", 0)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x7f0000000000

    def numel(self):
        return self.shape.numel()


@pytest.mark.parametrize("stream", [None, 5, 9])
def test_results_are_made_on_the_stream_of_the_call(streams, monkeypatch, stream):
    """In the order of its work: the zeros behind a cache read's lengths above all,
    which another stream would write at any time, over the rows that were read."""
    import online_activation_aware_ttq_amd as ttq
    made = []

    def make(shape, dtype=None, device=None):
        made.append(streams.now)
        return Fake(shape, dtype)

    monkeypatch.setattr(torch, "empty", make)
    monkeypatch.setattr(torch, "zeros", make)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(_binding, "_enqueue", lambda *a: None)
    monkeypatch.setenv("TTQ_INJECT_HIP_ERROR", "1")  # for those that call the library directly
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    X, codes, s = Fake((3, 64), bf), Fake((8, 32), u8), Fake((8, 2), f32)
    kw = dict(bits=4, group=32, stream=stream)
    ttq.ttq_cache_read(codes, s, s, Fake((1, 2), i32), Fake((1,), i32), page_tokens=4, **kw)
    ttq.ttq_adapters(X, Fake((2, 8, 64), bf), Fake((2, 16, 8), bf), Fake((3,), i32), stream=stream)
    ttq.ttq_moe(X, Fake((2, 64), bf), Fake((2, 128, 32), u8), Fake((2, 128, 2), f32),
                Fake((2, 128, 2), f32), Fake((2, 64), f32), Fake((2, 64, 32), u8), Fake((2, 64, 2), f32),
                Fake((2, 64, 2), f32), Fake((2, 64), f32), top_k=1, **kw)
    with pytest.raises(ttq.TTQError):
        ttq.ttq_qmatmul(codes, s, s, Fake((64,), f32), X, **kw)
    with pytest.raises(ttq.TTQError):
        ttq.ttq_quantize(Fake((8, 64), bf), X, p=2.0, lam=0.0, alpha=0.5, **kw)
    with pytest.raises(ttq.TTQError):
        ttq.ttq_linear(Fake((8, 64), bf), X, p=2.0, lam=0.0, alpha=0.5, **kw)
    assert len(made) >= 8 and set(made) == {stream or 5}
