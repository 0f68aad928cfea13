"""The binding's memory of gradient lists on the CPU, with stand-ins for torch's
allocations and streams: what a list that is dropped with calls queued on
other streams holds on to, and that no stream but the current one is ever
asked for anything (a caller's may have been destroyed)."""
import gc
import types

import pytest
import torch

import bucketed_gradient_all_amd as ddp

HOME, OTHER = 0x7000, 0x9000


class Allocation:
    device = "cuda:0"

    def __init__(self, at):
        self.at = at

    def data_ptr(self):
        return self.at

    def numel(self):
        return 64

    def record_stream(self, stream):
        raise AssertionError("a stream was recorded: it may be gone when the memory is freed")


@pytest.fixture
def device(monkeypatch):
    """Torch's streams and synchronizations as a log."""
    log = []

    def external(*a, **k):
        raise AssertionError("a bare handle was made a stream")

    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=HOME))
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda d=None: log.append(d))
    monkeypatch.setattr(ddp, "_parked", [], raising=False)
    return log


def _list_used_on(*streams):
    g = ddp.Grads(0)
    g.own(Allocation(0x100), Allocation(0x200))
    for s in streams:
        g.used_on(s)
    return g


@pytest.mark.parametrize("stream", [OTHER, 0, 1, 2])
@pytest.mark.parametrize("destroy", [False, True])
def test_memory_used_on_another_stream_waits_for_the_device(device, stream, destroy):
    g = _list_used_on(HOME, stream, stream)
    held = [g.workspace, g.scratch]
    if destroy:
        ddp.ddp_grads_destroy(g)
    del g
    gc.collect()
    assert ddp._parked == held and device == []
    ddp._free_parked()
    assert ddp._parked == [] and device == ["cuda:0"]
    ddp._free_parked()
    assert device == ["cuda:0"]   # nothing to wait for


def test_memory_used_on_its_own_stream_alone_is_freed_at_once(device):
    g = _list_used_on(HOME, HOME)
    del g
    gc.collect()
    assert ddp._parked == [] and device == []


@pytest.mark.parametrize("streams,parks", [((0, 1), False), ((1,), False), ((2,), True), ((OTHER,), True)])
def test_the_null_stream_has_two_names(device, monkeypatch, streams, parks):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=0))
    g = _list_used_on(*streams)
    del g
    gc.collect()
    assert bool(ddp._parked) == parks


def test_a_list_without_memory_of_its_own_parks_nothing(device):
    g = ddp.Grads(0)
    g.used_on(OTHER)
    del g
    gc.collect()
    assert ddp._parked == []


def test_memory_parked_while_the_device_drains_stays(device, monkeypatch):
    late = Allocation(0x300)

    def drain(d=None):
        device.append(d)
        ddp._parked.append(late)   # another list is dropped meanwhile

    monkeypatch.setattr(torch.cuda, "synchronize", drain)
    g = _list_used_on(OTHER)
    del g
    gc.collect()
    ddp._free_parked()
    assert ddp._parked == [late]


def test_a_failed_wait_frees_nothing(device, monkeypatch):
    def fail(d=None):
        raise RuntimeError("no")

    g = _list_used_on(OTHER)
    held = [g.workspace, g.scratch]
    del g
    gc.collect()
    monkeypatch.setattr(torch.cuda, "synchronize", fail)
    with pytest.raises(RuntimeError):
        ddp._free_parked()
    assert ddp._parked == held


def test_a_reducers_list_is_served_by_the_reducers_library(monkeypatch):
    """Another library loaded since knows nothing of the list."""
    calls = []

    class Library:
        def __init__(self, name):
            self.name = name

        def __getattr__(self, fn):
            def call(*a):
                calls.append((self.name, fn))
                if fn == "ddp_grads_from_reducer":
                    a[3]._obj.value = 0x1234
                return 0
            return call

    old, new = Library("old"), Library("new")
    monkeypatch.setattr(ddp, "_lib", new)
    g = ddp.ddp_grads_from_reducer(types.SimpleNamespace(handle=1, _lib=old), 0x100, 64)
    ddp.ddp_clip_grads(g, 1.0, 0x200, 0)
    del g
    gc.collect()
    assert calls == [("old", "ddp_grads_from_reducer"), ("old", "ddp_clip_grads"), ("old", "ddp_grads_destroy")]
