"""What the optimizer's objects do about streams when they are built (CPU only: the streams are stand-ins)."""
import pytest
import torch

from gradient_sync_amd import training as T


class Stream:
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
