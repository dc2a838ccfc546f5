"""Which stream the workspace of a product belongs to (no GPU: a fake of the
allocator's streams)."""

import contextlib
import ctypes

import pytest
import torch

import fully_sharded_amd as F
from fully_sharded_amd import products


class Side:
    """A stream by its handle, as torch's are."""

    def __init__(self, handle, log=None):
        self.cuda_stream = handle
        self.log = log

    def synchronize(self):
        self.log.append(("waited", self.cuda_stream))


@pytest.fixture
def log(monkeypatch):
    """What happens, in order: ("allocated", stream), ("waited", stream) and
    ("called", stream); the current stream is 7 on entry."""
    events, current = [], [7]

    @contextlib.contextmanager
    def stream(s):
        current.append(s.cuda_stream)
        yield
        current.pop()

    def empty(n, dtype, device):
        events.append(("allocated", current[-1]))
        return torch.zeros(n, dtype=dtype)

    def bound(name, args, keep, tensors):
        def run(s=None):
            on = current[-1] if s is None else getattr(s, "cuda_stream", None) or s.value
            events.append(("called", on))
        run.call = None
        return run
    monkeypatch.setattr(torch.cuda, "Stream", Side)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Side)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: Side(current[-1], events))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda _, s: events.append(("kept for", s.cuda_stream)))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda _: current[-1],
                        raising=False)
    monkeypatch.setattr(products, "_matrix", lambda t, *_: ctypes.c_void_p(t.data_ptr()))
    monkeypatch.setattr(products._b, "_dev", lambda t, _: t.data_ptr())
    monkeypatch.setattr(products, "_bound", bound)
    a, b = torch.zeros(9000, 64, dtype=torch.bfloat16), torch.zeros(9000, 64, dtype=torch.bfloat16)
    c = torch.zeros(64, 64)
    monkeypatch.setattr(torch, "empty", empty)
    return events, (a, b, c)


@pytest.mark.parametrize("stream", [None, Side(9), ctypes.c_void_p(9)])
def test_a_workspace_is_its_callers_streams(log, stream):
    events, operands = log
    F.fsdp_grouped_matmul("tn", *operands, stream=stream)
    on = 7 if stream is None else 9
    assert events == [("allocated", on), ("called", on)]


def test_a_kept_workspace_is_free_for_any_stream(log):
    """What may still use the memory is over when the binding is there."""
    events, operands = log
    f = F.bind_grouped_matmul("tn", *operands)
    assert events == [("allocated", 7), ("waited", 7)]
    f(Side(9))
    assert events[2] == ("called", 9)


def test_a_kept_workspace_outlives_its_calls(log):
    """A binding that nobody has any more leaves its workspace to the allocator:
    to be handed out again when the calls of every stream are done.  (Calls on the
    stream that it is of are in order with what comes next there.)"""
    events, operands = log
    f = F.bind_grouped_matmul("tn", *operands)
    for s in (None, Side(9), ctypes.c_void_p(9), ctypes.c_void_p(11), Side(9), None):
        f(s)
    with torch.cuda.stream(Side(13)):
        f()
    assert [e for e in events if e[0] == "kept for"] == [("kept for", s) for s in (9, 11, 13)]


def test_no_workspace_no_wait(log):
    events, (a, b, c) = log
    f = F.bind_grouped_matmul("tn", a[:100], b[:100], c)
    f()
    given = torch.zeros(1 << 20, dtype=torch.uint8)
    F.bind_grouped_matmul("tn", a, b, c, workspace=given)
    assert events == [("called", 7)]
