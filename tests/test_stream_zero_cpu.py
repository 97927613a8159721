"""The default stream's handle is 0, which torch.cuda.ExternalStream takes for none given: it hands out a stream of its
pool. No GPU: stream objects are stand-ins."""
import contextlib

import pytest
import torch

import adamw_hybrid_optimizer_muon_b200 as ma


@pytest.fixture
def streams(monkeypatch):
    """What torch was asked for, in order."""
    asked = []

    class Stream:
        def __init__(self, name):
            self.name = name

        def record_event(self, event=None):
            asked.append(("event", self.name))

        def wait_event(self, event):
            asked.append(("wait", self.name))

    class Event:
        def __init__(self, **kw):
            pass

        def record(self, stream):
            asked.append(("event", stream.name))

    @contextlib.contextmanager
    def on(stream):
        asked.append(("on", stream.name))
        yield

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "Event", Event)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle or "one of the pool"))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream("default"))
    monkeypatch.setattr(torch.cuda, "stream", on)
    return asked


def test_allocations_and_copies_for_the_default_stream(streams):
    with ma._on_stream(0):
        pass
    with ma._on_stream(4096):
        pass
    assert streams == [("on", "default"), ("on", 4096)]


def test_sums_on_the_default_stream_and_another(streams, monkeypatch):
    handles = iter([0, 0, 4096, 0])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: next(handles))
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False)
    monkeypatch.setattr(ma, "_LAST_SUM", {})
    monkeypatch.setattr(ma, "_SUM_STREAMS", {-1: {4096: torch.cuda.ExternalStream(4096)}})
    for _ in range(4):
        ma._sum_in_turn(-1, lambda: None)
    assert streams == [("event", "default"), ("event", "default"), ("wait", 4096), ("event", 4096), ("wait", "default"),
                       ("event", "default")]


def test_host_copies_on_the_default_stream(streams):
    class Plan:
        def step_from_host(self, *args):
            streams.append(("copies", args[-1]))

    opt = object.__new__(ma.MuonAdamW)
    opt._plan, opt._clip, opt.groups, opt.step_count, opt.entries = Plan(), None, [], 0, []
    opt._ensure_plan = lambda grads: None
    opt._set_clip = lambda max_norm, grad_scale: None
    opt.step_from_host([], [], copy_stream=0)
    opt.step_from_host([], [], copy_stream=4096)
    assert streams == [("copies", 0), ("event", "default"), ("copies", 4096), ("event", 4096)]
