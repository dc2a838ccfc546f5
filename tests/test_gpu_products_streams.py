"""The workspaces that the products' binding allocates, by torch's allocator:
each belongs to the stream that uses it, or is free for all of them."""

import ctypes

import pytest
import torch

import fully_sharded_amd as F
from fully_sharded_amd import products

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _gpu(request):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    F.lib()
    print(f"[gpu] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def operands():
    a = (torch.arange(9000 * 64, device=DEV) % 7 - 3).view(9000, 64).bfloat16()
    b = (torch.arange(9000 * 72, device=DEV) % 5 - 2).view(9000, 72).bfloat16()
    return a, b, torch.zeros(64, 72, device=DEV), (a.double().T @ b.double()).float()


def stream_of(t):
    """The stream whose pool a tensor's memory is of."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's")


@pytest.mark.parametrize("handle", [False, True])
def test_a_workspace_is_of_the_calls_stream(monkeypatch, handle):
    a, b, c, want = operands()
    of, plain = [], products._plain

    def watch(op, a, b, c, offsets, accumulate, workspace):
        of.append(stream_of(workspace))
        return plain(op, a, b, c, offsets, accumulate, workspace)
    monkeypatch.setattr(products, "_plain", watch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    F.fsdp_grouped_matmul("tn", a, b, c,
                          stream=ctypes.c_void_p(side.cuda_stream) if handle else side)
    torch.cuda.current_stream().wait_stream(side)
    assert of == [side.cuda_stream]
    assert torch.equal(c, want)
    c.zero_()
    F.fsdp_grouped_matmul("tn", a, b, c)
    assert of[1] == torch.cuda.current_stream().cuda_stream
    assert torch.equal(c, want)


def test_a_binding_waits_for_its_workspace():
    """The current stream is busy when the call is bound; then it is not, and the
    call runs on another one at once."""
    a, b, c, want = operands()
    x = torch.randn(4096, 4096, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(30):
        y = x @ x
    assert not torch.cuda.current_stream().query()
    f = F.bind_grouped_matmul("tn", a, b, c)
    assert torch.cuda.current_stream().query()
    f(side)
    side.synchronize()
    assert torch.equal(c, want) and y.shape == x.shape


def test_a_dropped_bindings_workspace_waits_for_its_calls():
    """Its memory is not handed out while a call on another stream may use it."""
    a, b, c, want = operands()
    side = torch.cuda.Stream()
    x = torch.randn(4096, 4096, device=DEV)
    ws = F.grouped_matmul_workspace("tn", a, b, c)
    n = ws.numel()
    del ws
    torch.cuda.synchronize()
    f = F.bind_grouped_matmul("tn", a, b, c)
    where = f.call._keep[-1].data_ptr()
    assert f.call._keep[-1].numel() == n
    with torch.cuda.stream(side):
        for _ in range(30):
            y = x @ x
    f(side)
    del f
    new = torch.empty(n, dtype=torch.uint8, device=DEV)
    assert not side.query()
    assert not new.data_ptr() <= where < new.data_ptr() + n
    side.synchronize()
    assert torch.equal(c, want) and y.shape == x.shape


def test_bound_while_captured():
    """No wait then (a capture forbids it): the graph's own memory."""
    a, b, c, want = operands()
    F.fsdp_grouped_matmul("tn", a, b, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = F.bind_grouped_matmul("tn", a, b, c)
        f()
    for _ in range(3):
        c.zero_()
        torch.cuda.synchronize()
        graph.replay()
        assert torch.equal(c, want)
