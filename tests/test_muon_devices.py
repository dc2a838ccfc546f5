"""The Muon binding's checks of devices, streams and workspace types (no GPU:
what it asks torch of the devices is replaced, and no call gets past the
library's checks)."""

import ctypes
from types import SimpleNamespace

import pytest
import torch

import fully_sharded_amd as F
from fully_sharded_amd import muon


def on(device):
    return SimpleNamespace(device=SimpleNamespace(index=device))


@pytest.fixture
def current(monkeypatch):
    """The current device, as torch tells it; set now[0] to change it."""
    now = [0]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    return now


def stream(device):
    return SimpleNamespace(device=SimpleNamespace(index=device), cuda_stream=0)


def test_tensors_on_another_device_are_refused(current):
    muon._caller("fsdp_muon_prepare", (), (on(0), on(0)))
    for tensors in ((on(1),), (on(0), on(1))):
        with pytest.raises(ValueError, match="current device"):
            muon._caller("fsdp_muon_prepare", (), tensors)


def test_a_bound_call_is_refused_where_another_device_is_current(current):
    _, go = muon._caller("fsdp_muon_prepare", (), (on(0),))
    with pytest.raises(F.FsdpError):    # of no handle: the library was called
        go((None,), None)
    current[0] = 1
    with pytest.raises(ValueError, match="current device"):
        go((None,), None)
    with pytest.raises(ValueError, match="current device"):
        go((None,), stream(0))


def test_a_stream_of_another_device_is_refused(current):
    current[0] = 1
    _, go = muon._caller("fsdp_muon_prepare", (), (on(1),))
    for s in (stream(1), ctypes.c_void_p(0), None):
        with pytest.raises(F.FsdpError):
            go((None,), s)
    with pytest.raises(ValueError, match="stream"):
        go((None,), stream(0))


def test_workspace_types_are_those_of_the_tensors():
    """bf16 bits in 16-bit integers are taken wherever tensors of them are;
    anything else is refused as such a tensor is."""
    mu = F.Muon(F.Plan([(60, 70)], 2, "flat"))
    want = mu.workspace_bytes(torch.bfloat16, torch.bfloat16)
    for t in (torch.int16, torch.uint16):
        assert mu.workspace_bytes(t, t) == want
        assert mu.workspace(t, t, device="cpu").numel() == want[0]
    for t in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(TypeError, match="dtype"):
            mu.workspace_bytes(t, torch.bfloat16)
        with pytest.raises(TypeError, match="dtype"):
            mu.workspace(torch.float32, t, device="cpu")
