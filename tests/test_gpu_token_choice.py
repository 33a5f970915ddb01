"""What depends on a token's own choice, together as a layer uses it: a linear with
the adapters of its users, the router's product, the choice of experts and the
experts.  Every step is checked on the inputs that it got; the whole also as a
captured graph, at once with another one, and with weights streamed ahead."""
import numpy as np
import pytest
import torch

import exl3_synth as synth
import oracle
import trellis_quantized_gb300 as tq
from gpu_util import assert_close, dev, host
from test_gpu_adapters import _check, _i32, _large, _pool, _reference, _starts
from test_gpu_router import W_TOL, _check_logits, _route_exact

pytestmark = pytest.mark.gpu

HIDDEN, INTER, E, TOPK = 512, 256, 16, 4


class Layer:
    """x -> linear + adapters -> norm -> logits -> ids, weights -> experts.  (The norm is a
    layer's own: the linear's outputs have a magnitude of sqrt(512), whose products in
    the experts pass fp16's range.)"""

    def __init__(self, T, seed=0):
        self.T, self.R = T, 24 if T < 2000 else 128
        assert _large(T, self.R, HIDDEN) == (T > 2000)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.moe = synth.moe_case(60, seed, T, E=E, topk=TOPK, hidden=HIDDEN, inter=INTER, K=4)
        m = self.moe
        self.keep = [dev(a) for a in (m.w13.trellis, m.w13.suh, m.w13.svh, m.w2.trellis, m.w2.suh, m.w2.svh)]
        self.w13 = tq.expert_proj(*self.keep[:3], m.w13.K)
        self.w2 = tq.expert_proj(*self.keep[3:], m.w2.K)
        self.lin = synth.linear_case(61, seed, T, HIDDEN, HIDDEN, 4)
        self.x = dev(self.lin.x)
        self.weights = [dev(a) for a in (self.lin.trellis, self.lin.suh, self.lin.svh)]
        self.pool = _pool(4, self.R, HIDDEN, HIDDEN, seed=seed)
        self.adapters = tq.adapters(*self.pool)
        self.rows = [T] if T < 3 else [T // 3, 1, T - T // 3 - 1]
        self.users = [2, -1, 0][:len(self.rows)]
        self.q_start, self.ids_of = _i32(_starts(self.rows)), _i32(self.users)
        self.plan = tq.exl3_adapter_plan(self.q_start, self.ids_of, T, 4)
        w = torch.randn((E, HIDDEN), generator=g, device="cuda") / HIDDEN ** 0.5
        self.w_router = w
        self.router = tq.router(w)
        self.bias = 0.05 * torch.randn(E, generator=g, device="cuda")
        self.rule = tq.route_rule(TOPK, score=tq.EXL3_SCORE_SIGMOID, bias=self.bias, groups=4, groups_kept=2,
                                  group_score=tq.EXL3_GROUP_TOP2, scale=2.0)
        f16 = dict(dtype=torch.float16, device="cuda")
        self.y0, self.y, self.n, self.z = (torch.empty((T, HIDDEN), **f16) for _ in range(4))
        self.logits = torch.empty((T, E), device="cuda")
        self.ids = torch.empty((T, TOPK), dtype=torch.int32, device="cuda")
        self.w = torch.empty((T, TOPK), device="cuda")

    def step(self):
        tq.exl3_adapter_plan(self.q_start, self.ids_of, self.T, 4, plan=self.plan)
        tq.exl3_linear(self.x, *self.weights, 4, y=self.y0)
        tq.exl3_adapter_add(self.x, self.y0, self.adapters, self.plan, out=self.y)
        self.n.copy_(self.y.float() * torch.rsqrt(self.y.float().square().mean(-1, keepdim=True)))
        tq.exl3_router_logits(self.n, self.router, logits=self.logits)
        tq.exl3_route(self.logits, self.rule, ids=self.ids, weights=self.w)
        tq.exl3_moe_grouped(self.n, self.ids, self.w, self.w13, self.w2, E, y=self.z)

    def outputs(self):
        return [t.clone() for t in (self.y0, self.y, self.logits, self.ids, self.w, self.z)]


@pytest.mark.parametrize("T", [1, 12, 300])
def test_a_layers_choices(T):
    l = Layer(T)
    l.step()
    torch.cuda.synchronize()
    assert_close(host(l.y0), oracle.linear(host(l.x).view(np.uint16), l.lin.trellis, l.lin.suh, l.lin.svh, 4), "linear")
    _check(l.y, *_reference(l.x.view(torch.float16), l.y0, l.pool, l.rows, l.users))
    _check_logits(l.n, l.w_router, None, l.logits)
    ids, w = _route_exact(l.logits, TOPK, "sigmoid", l.bias, 4, 2, "top2", True, 2.0)
    assert torch.equal(l.ids.long(), ids) and ((l.w.double() - w).abs() <= W_TOL * w).all()
    m = l.moe
    ref = oracle.moe(host(l.n).view(np.uint16), host(l.ids), host(l.w), m.w13.trellis, m.w13.suh, m.w13.svh, m.w13.K,
                     m.w2.trellis, m.w2.suh, m.w2.svh, m.w2.K)
    assert_close(host(l.z), ref, "experts")


@pytest.mark.parametrize("T", [1, 12, 300, 2500])
def test_a_graph_gives_the_same_bits(T):
    l = Layer(T)
    l.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        l.step()
    users = [[2, -1, 0], [1, 1, 3], [-1, 0, -1]]
    for u in users:
        l.ids_of.copy_(_i32(u[:len(l.rows)]))
        l.step()
        torch.cuda.synchronize()
        want = l.outputs()
        for t in (l.y0, l.y, l.logits, l.ids, l.w, l.z):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(l.outputs(), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T", [40, 300, 2500])
def test_two_graphs_at_once(T):
    """Two captured layers replayed on two streams: nothing of one shows in the other.
    (The linears and experts take the stream's workspace, which graphs would share: here only what is new runs.)"""
    layers = [Layer(T, seed=s) for s in (1, 2)]

    def step(l):
        tq.exl3_adapter_add(l.x.view(torch.float16), l.y0, l.adapters, l.plan, out=l.y)
        tq.exl3_router_logits(l.n, l.router, logits=l.logits)
        tq.exl3_route(l.logits, l.rule, ids=l.ids, weights=l.w)

    graphs, want = [], []
    for l in layers:
        l.step()
        step(l)
        torch.cuda.synchronize()
        want.append(l.outputs())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(4):
                step(l)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for l, w in zip(layers, want):
        for a, b in zip(l.outputs(), w):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T", [12, 300, 2500])
def test_one_workspace_for_all_calls(T):
    """Every operator in one workspace, whose counters the linears and experts find at zero."""
    l = Layer(T)
    l.step()
    torch.cuda.synchronize()
    want = l.outputs()
    need = max(tq.exl3_linear_workspace_size(T, HIDDEN, HIDDEN, 4), tq.exl3_adapter_add_workspace_size(T, l.R),
               tq.exl3_router_logits_workspace_size(), tq.exl3_moe_workspace_size(T, TOPK, E, l.w13, l.w2))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    kw = dict(workspace_buf=ws)
    for _ in range(3):
        tq.exl3_linear(l.x, *l.weights, 4, y=l.y0, **kw)
        tq.exl3_adapter_add(l.x.view(torch.float16), l.y0, l.adapters, l.plan, out=l.y, **kw)
        tq.exl3_router_logits(l.n, l.router, logits=l.logits, **kw)
        tq.exl3_moe_grouped(l.n, l.ids, l.w, l.w13, l.w2, E, y=l.z, **kw)
    torch.cuda.synchronize()
    assert tq.exl3_check_device_error(ws) == 0
    for a, b in zip(l.outputs(), want):
        assert torch.equal(a, b)


def test_with_weights_streamed_ahead():
    """One-row linears that stream their weights during the kernel ahead of them."""
    l = Layer(1)
    l.step()
    torch.cuda.synchronize()
    want = l.outputs()
    before = tq.exl3_set_weight_prefetch(True)
    try:
        for _ in range(5):
            l.step()
        torch.cuda.synchronize()
        for a, b in zip(l.outputs(), want):
            assert torch.equal(a, b)
    finally:
        tq.exl3_set_weight_prefetch(before)
