"""What the optimizer's objects do about streams when they are built (CPU only: the streams are stand-ins)."""
import pytest
import torch

from gradient_sync_amd import training as T


class Stream:
    cuda_stream = 7

    def __init__(self, log):
        self.log = log

    def synchronize(self):
        self.log.append("synchronize")


@pytest.fixture
def log(monkeypatch):
    log = []
    zeros = torch.zeros

    def filled(*shape, device=None, **kw):
        log.append("fill")
        return zeros(*shape, **kw)
    monkeypatch.setattr(T, "_list", lambda ts, *a, **kw: list(ts))
    monkeypatch.setattr(T.torch, "zeros", filled)
    monkeypatch.setattr(T.torch.cuda, "current_stream", lambda device=None: Stream(log))
    monkeypatch.setattr(T.torch.cuda, "is_current_stream_capturing", lambda: "capture" in log)
    return log


def make():
    g = [torch.ones(5)]
    return T.GradNorm(g, T.StepCtrl(device="cpu"))


def test_the_norms_workspace_is_zeroed_before_it_can_run_on_any_stream(log):
    make()
    assert log == ["fill", "synchronize"]


def test_a_norm_built_while_its_stream_captures_does_not_wait(log):
    log.append("capture")
    make()
    assert log == ["capture", "fill"]


def test_a_norm_that_runs_once_on_its_own_stream_does_not_wait(log, monkeypatch):
    monkeypatch.setattr(T.GradNorm, "run", lambda self, *a: self.ctrl)
    T.dp_grad_norm([torch.ones(5)], T.StepCtrl(device="cpu"))
    assert log == ["fill"]


def test_a_norms_memory_is_kept_for_every_stream_it_runs_on(log, monkeypatch):
    class Memory:
        def __init__(self, name):
            self.name = name

        def record_stream(self, s):
            log.append((self.name, s))

        def data_ptr(self):
            return 256

    class Library:
        @staticmethod
        def dp_grad_norm(*args):
            log.append(("run", args[-1]))
            return 0
    class Given:
        def __init__(self, handle, number):
            self.cuda_stream, self.stream_id = handle, number
    monkeypatch.setattr(T, "lib", lambda: Library)
    monkeypatch.setattr(T, "_at", lambda stream: stream if isinstance(stream, int) else stream.cuda_stream)
    norm = make()
    monkeypatch.setattr(T.torch.cuda, "Stream", Given)
    norm.workspace, norm.ctrl.buf = Memory("workspace"), Memory("ctrl")
    del log[:]
    home, side, default, foreign = Given(7, 1), Given(9, 3), Given(0, 0), Given(11, 11)
    for stream in (home, side, side, default, foreign, 13, home):
        norm.run(1.0, stream=stream)
    assert log == [("run", 7), ("workspace", side), ("ctrl", side), ("run", 9), ("run", 9),
                   ("workspace", default), ("ctrl", default), ("run", 0), ("run", 11), ("run", 13), ("run", 7)]


@pytest.mark.parametrize("handle", [0, 9, 1 << 47])
def test_a_streams_handle_is_a_number(handle):
    assert T._at(handle) == handle
