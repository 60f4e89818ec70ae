"""Scratch that a call allocates on torch's current stream for kernels on another one is kept for that one, the default
stream among them. Without a GPU: streams and the tensor are stand-ins."""
import pytest

torch = pytest.importorskip("torch")
import quantized_weight_gguf_gb300 as q  # noqa: E402


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Buffer:
    device = "cuda:0"

    def __init__(self):
        self.kept_for = []

    def record_stream(self, s):
        self.kept_for.append(s.cuda_stream)


@pytest.fixture()
def current(monkeypatch):
    now = Stream(0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle))
    return now


@pytest.mark.parametrize("now,stream,kept", [
    (0, None, []), (0, 0, []), (0, 7, [7]), (0, Stream(7), [7]), (7, 0, [0]), (7, Stream(0), [0]), (7, 7, []),
    (7, Stream(7), []), (7, 9, [9])])
def test_kept_for_the_stream_that_uses_it(current, now, stream, kept):
    current.cuda_stream = now
    buf = Buffer()
    q._keep_until_done(buf, stream)
    assert buf.kept_for == kept
    q._keep_until_done(None, stream)
