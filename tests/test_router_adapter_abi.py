"""Host side of routing and adapters, without a GPU: refusals (every call below
is rejected before anything is launched), plan sizes and the bindings' checks."""
import ctypes
import math

import pytest
import torch

import trellis_quantized_gb300 as tq

FAKE = ctypes.c_void_p(0x10000)       # 256-byte aligned, never dereferenced
FAKE_MIS = ctypes.c_void_p(0x10008)   # 8-byte aligned
FAKE_ODD = ctypes.c_void_p(0x10001)


def _err():
    return tq.lib().exl3_last_error().decode()


ref = lambda s: None if s is None else ctypes.byref(s)


def _fill(cls, base, kw):
    d = dict(base)
    d.update(kw)
    return cls(*[d[n] for n, _ in cls._fields_])


def _logits(r="default", **kw):
    g = lambda n, v: kw.pop(n, v)
    call = dict(x=g("x", FAKE), xs=g("xs", 2048), T=g("T", 3), out=g("out", FAKE), ws=g("ws", FAKE), wsb=g("wsb", 256))
    if r == "default":
        r = _fill(tq.Router, dict(w=FAKE.value, w_scale=None, bias=None, E=256, k=2048), kw)
    return tq.lib().exl3_router_logits(call["x"], call["xs"], call["T"], ref(r), call["out"], call["ws"], call["wsb"],
                                       None)


RULE = dict(score=0, bias=None, groups=1, groups_kept=1, group_score=0, topk=8, renormalise=1, scale=1.0)


def _route(r="default", **kw):
    g = lambda n, v: kw.pop(n, v)
    call = [g("l", FAKE), g("ls", 256), g("idt", 1), g("T", 3), g("E", 256)]
    out = [g("ids", FAKE), g("weights", FAKE)]
    if r == "default":
        r = _fill(tq.RouteRule, RULE, kw)
    return tq.lib().exl3_route(*call, ref(r), *out, None)


POOL = dict(a=FAKE.value, b=FAKE.value, scale=FAKE.value, rank=None, count=8, max_rank=16, k=2048, n=512)


def _add(p="default", **kw):
    g = lambda n, v: kw.pop(n, v)
    call = [g("x", FAKE), g("xs", 2048), g("y", FAKE), g("ys", 512), g("out", ctypes.c_void_p(0x20000)), g("os", 512),
            g("dt", 0)]
    tail = [g("plan", FAKE), g("T", 3), g("batch", 2), g("ws", FAKE), g("wsb", 1 << 30)]
    if p == "default":
        p = _fill(tq.Adapters, POOL, kw)
    return tq.lib().exl3_adapter_add(*call, ref(p), *tail, None)


def _plan(**kw):
    d = dict(qs=FAKE, ad=FAKE, T=3, batch=2, count=8, plan=FAKE, nbytes=1 << 30)
    d.update(kw)
    return tq.lib().exl3_adapter_plan(*d.values(), None)


A, S, W = tq.EXL3_ERR_ARG, tq.EXL3_ERR_SHAPE, tq.EXL3_ERR_WORKSPACE


@pytest.mark.parametrize("kw,code,text", [
    (dict(x=None), A, "x is NULL"), (dict(x=FAKE_MIS), A, "x is not"), (dict(out=None), A, "logits"),
    (dict(out=FAKE_MIS), A, "logits"), (dict(w=None), A, "router.w"), (dict(w=FAKE_MIS.value), A, "router.w"),
    (dict(w_scale=FAKE_ODD.value), A, "w_scale"), (dict(bias=FAKE_ODD.value), A, "bias"), (dict(E=0), S, "E ="),
    (dict(E=1025), S, "E ="), (dict(k=0), S, "k ="), (dict(k=2044), S, "k ="), (dict(xs=2040), S, "stride"),
    (dict(xs=2052), S, "stride"), (dict(xs=1 << 39), S, "stride"), (dict(T=-1), S, "T ="), (dict(T=(1 << 22) + 1), S, "T ="),
    (dict(ws=None), W, "workspace"), (dict(wsb=255), W, "workspace"),
])
def test_router_logits_refuses(kw, code, text):
    assert _logits(**kw) == code and text in _err()


def test_router_pack_refuses():
    L = tq.lib()
    for args, code in (((None, 8, 64, FAKE, FAKE), A), ((FAKE_MIS, 8, 64, FAKE, FAKE), A), ((FAKE, 8, 64, None, FAKE), A),
                       ((FAKE, 8, 64, FAKE, FAKE_ODD), A), ((FAKE, 0, 64, FAKE, FAKE), S), ((FAKE, 8, 60, FAKE, FAKE), S)):
        assert L.exl3_router_pack(*args, None) == code


@pytest.mark.parametrize("kw,code,text", [
    (dict(l=None), A, "logits"), (dict(l=ctypes.c_void_p(0x10002)), A, "logits"), (dict(ids=None), A, "ids"),
    (dict(ids=FAKE_ODD), A, "ids"), (dict(weights=None), A, "weights"), (dict(idt=2), A, "in_dtype"),
    (dict(T=-1), S, "T ="), (dict(E=0), S, "E ="), (dict(E=1025, ls=2000), S, "E ="), (dict(ls=255), S, "stride"),
    (dict(score=2), A, "score"), (dict(score=-1), A, "score"), (dict(group_score=2), A, "group_score"),
    (dict(renormalise=2), A, "renormalise"), (dict(scale=math.nan), A, "scale"), (dict(scale=math.inf), A, "scale"),
    (dict(bias=FAKE_ODD.value), A, "bias"), (dict(groups=0), S, "groups"), (dict(groups=3), S, "groups"),
    (dict(groups=64, groups_kept=64), S, "groups"), (dict(groups=8, groups_kept=0), S, "groups_kept"),
    (dict(groups=8, groups_kept=9), S, "groups_kept"), (dict(topk=0), S, "topk"), (dict(topk=33), S, "topk"),
    (dict(groups=32, groups_kept=1, topk=9), S, "topk"), (dict(E=4, ls=4, topk=5), S, "topk"),
])
def test_route_refuses(kw, code, text):
    assert _route(**kw) == code and text in _err()


@pytest.mark.parametrize("kw,code,text", [
    (dict(x=None), A, "x is NULL"), (dict(y=FAKE_MIS), A, "y is not"), (dict(out=None), A, "out"),
    (dict(plan=None), A, "plan"), (dict(plan=ctypes.c_void_p(0x10010)), A, "plan"), (dict(dt=2), A, "dtype"),
    (dict(ws=None), W, "workspace"), (dict(wsb=255), W, "workspace"), (dict(T=1000, wsb=1000 * 16 * 4), W, "needed"),
    (dict(xs=2040), S, "x: stride"), (dict(xs=2052), S, "x: stride"), (dict(ys=508), S, "y: stride"),
    (dict(os=516), S, "out: stride"), (dict(os=520, out=FAKE), S, "strides differ"), (dict(a=None), A, "adapters.a"),
    (dict(b=FAKE_MIS.value), A, "adapters.b"), (dict(scale=None), A, "scale"), (dict(rank=FAKE_ODD.value), A, "rank"),
    (dict(count=0), S, "count"), (dict(count=4097), S, "count"), (dict(max_rank=0), S, "max_rank"),
    (dict(max_rank=12), S, "max_rank"), (dict(max_rank=136), S, "max_rank"), (dict(k=2000), S, "k ="),
    (dict(n=64), S, "n ="), (dict(T=-1), S, "T ="), (dict(batch=0), S, "batch"),
])
def test_adapter_add_refuses(kw, code, text):
    assert _add(**kw) == code and text in _err()


@pytest.mark.parametrize("kw,code,text", [
    (dict(qs=None), A, "q_start"), (dict(ad=FAKE_ODD), A, "adapter"), (dict(T=-1), S, "T ="),
    (dict(batch=0), S, "batch"), (dict(batch=(1 << 20) + 1), S, "batch"), (dict(count=0), S, "count"),
    (dict(count=4097), S, "count"), (dict(plan=None), W, "workspace"), (dict(plan=FAKE_MIS), W, "aligned"),
    (dict(nbytes=256), W, "needed"),
])
def test_adapter_plan_refuses(kw, code, text):
    assert _plan(**kw) == code and text in _err()


def test_null_descriptors_are_refused():
    assert _logits(None) == A and _route(None) == A and _add(None) == A


def test_no_rows_enqueue_nothing():
    """T = 0 passes every check and launches nothing (the addresses are not real)."""
    assert _logits(T=0) == 0 and _route(T=0) == 0 and _add(T=0) == 0


@pytest.mark.parametrize("T,batch,count", [(1, 1, 1), (1, 64, 8), (4096, 4, 8), (7, 7, 4096), (130, 3, 2)])
def test_plan_size_holds_its_parts(T, batch, count):
    """Control block, a place per sequence and row, and 16 bytes for every tile
    that the rows can make: each adapter in use and the rows without one end in
    at most one part-filled tile."""
    used = min(T, batch, count) + 1
    tiles = min(T, T // 16 + used) + min(T, T // 128 + used)
    need = 256 + 4 * batch + 4 * T + 16 * tiles
    assert need <= tq.exl3_adapter_plan_size(T, batch, count) <= need + 5 * 256


def test_plan_size_of_refused_shapes_is_zero():
    assert all(tq.exl3_adapter_plan_size(*s) == 0 for s in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 4097), (1 << 23, 1, 1)))


def test_bindings_refuse_other_types():
    """bfloat16 has fp16's width and other values; host tensors have no device address."""
    w = torch.zeros(8, 64)
    with pytest.raises(TypeError, match="w must be"):
        tq.router(w.bfloat16())
    with pytest.raises(ValueError, match="CUDA"):
        tq.router(w.half())
    with pytest.raises(TypeError, match="a must be torch.float16"):
        tq.adapters(torch.zeros(2, 8, 128, dtype=torch.bfloat16), torch.zeros(2, 128, 8), torch.ones(2))
    with pytest.raises(ValueError, match="CUDA"):
        tq.route_rule(2, bias=torch.zeros(8))
    with pytest.raises(ValueError, match="CUDA"):
        tq.exl3_route(torch.zeros(2, 8), tq.route_rule(2))
    with pytest.raises(ValueError, match="CUDA"):
        tq.exl3_adapter_plan(torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 1, 1)


def test_descriptors_keep_the_sizes_of_their_tensors():
    """Kernels go by the descriptor's sizes, a call's checks by the tensors': they must not part.
    (Descriptors as router() and adapters() leave them, of addresses that nothing reads.)"""
    router, pool = tq.Router(FAKE.value, None, None, 16, 64), tq.Adapters(FAKE.value, FAKE.value, FAKE.value, None, 2, 8, 128, 256)
    for d in (router, pool):
        d.k = d.k                                          # (not made yet)
        d._address = ctypes.addressof(d)
    for d, names in ((router, "E k"), (pool, "count max_rank k n")):
        for name in names.split():
            before = getattr(d, name)
            with pytest.raises(AttributeError, match="size"):
                setattr(d, name, before + 128)
            assert getattr(d, name) == before
    router.bias = FAKE.value                               # an address may be set
    assert router.bias == FAKE.value


def test_workspaces_of_another_device_are_refused():
    class Elsewhere:                                       # what a tensor on the second GPU says of itself
        device = torch.device("cuda", 1)
        numel = element_size = lambda self: 256
        get_device = lambda self: 1

    tq_ptr, tq._ptr = tq._ptr, lambda t, name: FAKE
    try:
        assert tq._workspace_arg(Elsewhere(), 256, torch.device("cuda", 1), None, 0) == (FAKE, 256 * 256)
        with pytest.raises(ValueError, match="workspace is on cuda:1"):
            tq._workspace_arg(Elsewhere(), 256, torch.device("cuda", 0), None, 0)
    finally:
        tq._ptr = tq_ptr


def test_relaxing_captures_wants_a_place_for_the_mode():
    assert tq.lib().exl3_relax_capture(1, None) == A and "previous" in _err()


def _add_scratch(**kw):
    d = dict(T=3, k=2048, n=512, R=16, ws=FAKE, wsb=256, scratch=None, sb=0, plan=FAKE)
    d.update(kw)
    p = _fill(tq.Adapters, POOL, dict(k=d["k"], n=d["n"], max_rank=d["R"]))
    return tq.lib().exl3_adapter_add_scratch(FAKE, d["k"], FAKE, d["n"], ctypes.c_void_p(0x20000), d["n"], 0, ref(p), d["plan"],
                                             d["T"], 2, d["ws"], d["wsb"], d["scratch"], d["sb"], None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(ws=None), W, "workspace"), (dict(wsb=255), W, "workspace"), (dict(plan=None), A, "plan"),
    (dict(T=2000, R=128, n=4096), W, "scratch is NULL"), (dict(T=2000, R=128, n=4096, scratch=FAKE), W, "scratch has"),
    (dict(T=2000, R=128, n=4096, scratch=FAKE_MIS, sb=1 << 30), W, "aligned"), (dict(k=100), S, "k ="),
])
def test_adapter_add_scratch_refuses(kw, code, text):
    assert _add_scratch(**kw) == code and text in _err()


@pytest.mark.parametrize("T,R,n", [(47, 128, 17408), (48, 128, 17408), (63, 64, 41984), (2000, 16, 8448), (200, 8, 128),
                                   (1 << 22, 128, 1 << 20), (0, 16, 128)])
def test_scratch_sizes(T, R, n):
    """h of every row in two fp16 parts and a factor, where h passes from one kernel to another."""
    large = T >= 48 and T * (R + 16) ** 2 * n >= 1 << 34
    size, whole = tq.exl3_adapter_scratch_size(T, R, n), tq.exl3_adapter_add_workspace_size(T, R)
    assert (T * (4 * R + 4) <= size <= whole - 33024 < size + 256) if large else size == 0


def test_scratch_sizes_of_refused_shapes_are_zero():
    assert all(tq.exl3_adapter_scratch_size(*s) == 0 for s in ((-1, 16, 128), (1 << 23, 16, 128), (4096, 12, 4096), (4096, 128, 0)))
    assert _add_scratch(T=0) == 0
