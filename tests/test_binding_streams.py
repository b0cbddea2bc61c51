"""Which stream a call is given to, without a GPU: the binding's stream queries
are replaced by a machine of two GPUs whose current streams are set here."""
import contextlib
import types

import pytest
import torch

import group_limited_routing_sigmoid_amd as gl


def stream(dev, handle):
    return types.SimpleNamespace(device=torch.device("cuda", dev), cuda_stream=handle)


class Tensor:
    def __init__(self):
        self.used = []

    def record_stream(self, s):
        self.used.append(s)


@pytest.fixture
def two_gpus(monkeypatch):
    current = {0: 0, 1: 0}
    monkeypatch.setattr(gl, "_raw_stream", lambda dev: current[dev])
    monkeypatch.setattr(gl, "_current_device", lambda: 0)
    return current


def call(on, dev, t):
    got = []
    gl._run(lambda *a: got.append(a) or gl.OK, "call", on, dev, (t, None), 1, 2)
    return got[0]


def test_handed_to_its_stream(two_gpus):
    t = Tensor()
    assert call(True, 0, t) == (1, 2, 0) and t.used == []
    s = stream(0, 7)
    assert call(s, 0, t) == (1, 2, 7) and t.used == [s]
    two_gpus[0] = 7                                   # the current stream by another object
    assert call(stream(0, 7), 0, t) == (1, 2, 7) and t.used == [s]


@pytest.mark.parametrize("handle", [0, 7])
def test_stream_of_another_gpu_is_refused(two_gpus, handle):
    # also its default stream, whose handle every GPU shares
    with pytest.raises(ValueError, match="a stream of cuda:1 for tensors on cuda:0"):
        call(stream(1, handle), 0, Tensor())


def test_capture_is_asked_of_the_calls_own_stream(two_gpus, monkeypatch):
    # GPU 0 is current; a stream of GPU 1, and its current one, may be captured
    now = [stream(0, 0)]
    captured = set()

    @contextlib.contextmanager
    def on(s):
        now.append(s)
        yield
        now.pop()

    two_gpus[1] = 5
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: stream(d.index, two_gpus[d.index]))
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing",
                        lambda: (now[-1].device.index, now[-1].cuda_stream) in captured, raising=False)
    gpu = [torch.device("cuda", i) for i in range(2)]
    for where, want in ((set(), (False, False, False)), ({(0, 0)}, (True, False, False)),
                        ({(1, 5)}, (False, True, False)), ({(1, 9)}, (False, False, True))):
        captured.clear()
        captured.update(where)
        got = (gl._capturing(None, gpu[0]), gl._capturing(None, gpu[1]), gl._capturing(stream(1, 9), gpu[1]))
        assert got == want
