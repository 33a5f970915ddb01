"""The binding's own workspaces: kept by device and stream, and what captured graphs hold of them."""
import gc

import pytest
import torch

import trellis_quantized_gb300 as tq

pytestmark = pytest.mark.gpu


@pytest.fixture
def stream():
    """A stream that no workspace was asked for on (streams come from a pool and return)."""
    s = torch.cuda.Stream()
    for key in [k for k in tq._ws_cache if k[1] == s.cuda_stream]:
        del tq._ws_cache[key]
    return s


@pytest.mark.parametrize("named", [False, True])
def test_a_graphs_workspace_outlives_a_larger_one(stream, named):
    """A larger call takes the cached buffer's place; the graph's address stays allocated."""
    kw = dict(stream=stream) if named else {}
    with torch.cuda.stream(stream):
        address = tq.workspace(1 << 20, **kw).data_ptr()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            assert tq.workspace(1 << 20, **kw).data_ptr() == address
            torch.zeros(1, device="cuda")
        assert tq.workspace(3 << 20, **kw).data_ptr() != address
        gc.collect()
        again = [torch.empty(1 << 20, dtype=torch.uint8, device="cuda") for _ in range(64)]
        assert address not in [t.data_ptr() for t in again]


def test_outgrown_workspaces_are_bounded(stream):
    """Sizes that grow by little: each buffer is twice the one before it, and all before it no more than the last."""
    with torch.cuda.stream(stream):
        seen = {}
        for i in range(1, 200):
            ws = tq.workspace(4096 * i)
            assert ws.numel() >= 4096 * i and not ws.any()
            seen[ws.data_ptr()] = ws.numel()
        sizes = list(seen.values())
        assert len(sizes) < 10 and sum(sizes[:-1]) <= sizes[-1] < 4 * 4096 * 199


def test_memory_of_a_workspace_is_its_streams(stream):
    """What the current stream has freed, and may still be using, does not become another stream's workspace."""
    size = 5 << 20
    freed = torch.empty(size, dtype=torch.uint8, device="cuda")
    address = freed.data_ptr()
    del freed
    assert tq.workspace(size, stream=stream).data_ptr() != address
    again = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() == address                     # (it was there to be had)


def test_memory_of_plans_and_packed_weights_is_their_streams(stream):
    q, ids = torch.tensor([0, 900000], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    w = torch.randn((1024, 2048), device="cuda")
    for make, state in ((lambda: tq.exl3_adapter_plan(q, ids, 900000, 1, stream=stream), lambda p: p.data),
                        (lambda: tq.router(w, stream=stream), lambda r: r._keep[0])):
        torch.cuda.synchronize()
        held = state(make())                               # (of the same size: what is freed next would fit)
        size = held.numel() * held.element_size()
        freed = torch.empty(size, dtype=torch.uint8, device="cuda")
        address = freed.data_ptr()
        del freed
        assert state(make()).data_ptr() != address
        torch.cuda.synchronize()


def test_a_workspace_first_asked_for_in_a_capture_is_cleared(stream):
    """Zero for everyone, though nothing of the graph has run, and of memory that no graph's temporaries are written to."""
    size, g = 1 << 20, torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        used = torch.empty(size, dtype=torch.uint8, device="cuda")
        used.fill_(0x55)
        del used
    g.replay()
    torch.cuda.synchronize()
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2, pool=g.pool(), stream=stream):
        temporary = torch.full((2 * size,), 0x55, dtype=torch.uint8, device="cuda")
        del temporary
        ws = tq.workspace(size)
        y = ws[:16].clone()
    with torch.cuda.stream(stream):
        assert tq.workspace(size).data_ptr() == ws.data_ptr()
    assert not ws.any()
    for graph in (g, g2, g):
        graph.replay()
        torch.cuda.synchronize()
        assert not ws.any()
        if graph is g2:                                    # (y shares its memory with the first graph's temporary)
            assert not y.any()


def test_a_linear_captured_without_a_call_before(stream):
    """Its counters are zero in the graph and for a call outside of it."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    k, n, K = 2048, 2048, 4
    t = torch.randint(-2**15, 2**15, (k // 16, n // 16, 16 * K), generator=g, device="cuda").to(torch.int16)
    suh, svh = (torch.ones(d, dtype=torch.float16, device="cuda") for d in (k, n))
    x = torch.randn((5, k), generator=g, device="cuda").half()
    want = tq.exl3_linear(x, t, suh, svh, K)
    torch.cuda.synchronize()
    graph, y = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(graph, stream=stream):
        tq.exl3_linear(x, t, suh, svh, K, y=y)
    with torch.cuda.stream(stream):
        assert torch.equal(tq.exl3_linear(x, t, suh, svh, K), want)
        ws = tq.workspace(1)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert tq.exl3_check_device_error(ws) == 0


def test_a_stream_is_its_handle(stream):
    """Other libraries' stream objects: whatever has a cuda_stream."""
    class Handle:
        cuda_stream = stream.cuda_stream

    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    T, k, n, R = 300, 256, 8192, 128
    x = torch.randn((T, k), generator=g, device="cuda").half()
    y = torch.randn((T, n), generator=g, device="cuda")
    a = torch.randn((2, R, k), generator=g, device="cuda").half()
    b = torch.randn((2, n, R), generator=g, device="cuda").half()
    w = torch.randn((16, k), generator=g, device="cuda")
    ad = tq.adapters(a, b, torch.ones(2, device="cuda"))
    q, ids = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 70, T], [1, 0]))
    want = tq.exl3_adapter_add(x, y, ad, tq.exl3_adapter_plan(q, ids, T, 2), out=torch.empty_like(y))
    want_logits = tq.exl3_router_logits(x, tq.router(w))
    out, graph = torch.empty_like(y), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    kw = dict(stream=Handle())
    plan, router = tq.exl3_adapter_plan(q, ids, T, 2, **kw), tq.router(w, **kw)
    logits = tq.exl3_router_logits(x, router, **kw)
    tq.exl3_adapter_add(x, y, ad, plan, out=out, **kw)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(logits, want_logits)
    with torch.cuda.graph(graph, stream=stream):
        tq.exl3_adapter_add(x, y, ad, plan, out=out, **kw)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_device_too_full_for_twice_the_size(stream, monkeypatch):
    """Then the size that was asked for has to do."""
    empty, asked = torch.empty, []

    def full(size, **kw):
        asked.append(size)
        if size > 3 << 20:
            raise torch.OutOfMemoryError("full")
        return empty(size, **kw)

    with torch.cuda.stream(stream):
        first = tq.workspace(2 << 20)
        monkeypatch.setattr(torch, "empty", full)
        ws = tq.workspace(3 << 20)
        assert asked == [4 << 20, 3 << 20] and ws.numel() == 3 << 20 and not ws.any()
        with pytest.raises(torch.OutOfMemoryError):
            tq.workspace(5 << 20)
        assert tq.workspace(1).data_ptr() == ws.data_ptr() != first.data_ptr()
