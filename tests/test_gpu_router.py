"""exl3_router_pack, exl3_router_logits and exl3_route against their definitions in 64 bits."""
import math

import pytest
import torch

import trellis_quantized_gb300 as tq

pytestmark = pytest.mark.gpu


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------- product

def _inputs(T, k, E, fp32, seed=0):
    g = _gen(seed)
    x = torch.randn((T, k), generator=g, device="cuda").half()
    w = torch.randn((E, k), generator=g, device="cuda") / math.sqrt(k)
    return x, w if fp32 else w.half()


def _check_logits(x, w, bias, got):
    """A sum of k products (fp16 by fp16 is exact in fp32) has at most k roundings
    of one fp32 unit of what was summed so far, itself at most sum |x w|; packed
    weights add 2^-22 of each product, the bias one more rounding."""
    xd, wd = x.double(), w.double()
    want = xd @ wd.t()
    size = xd.abs() @ wd.abs().t()
    tol = size * (x.shape[1] * 2.0 ** -23 + (2.0 ** -22 if w.dtype == torch.float32 else 0))
    if bias is not None:
        want = want + bias.double()
        tol = tol + want.abs() * 2.0 ** -24
    assert got.dtype == torch.float32 and torch.isfinite(got).all()
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("T", [1, 2, 3, 7, 8, 9, 48, 127, 128, 129, 1333])
@pytest.mark.parametrize("k,E", [(2048, 256), (128, 8), (5120, 60), (520, 1), (64, 5), (1048, 300)])
def test_logits(T, k, E, fp32):
    x, w = _inputs(T, k, E, fp32)
    got = tq.exl3_router_logits(x, tq.router(w))
    _check_logits(x, w, None, got)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("T,k,E", [(1, 256, 1024), (20, 256, 1024), (300, 8, 17), (5, 8, 17), (4096, 2048, 256),
                                   (3000, 1024, 512), (20000, 512, 64)])
def test_logits_with_bias(T, k, E, fp32):
    x, w = _inputs(T, k, E, fp32, seed=1)
    bias = torch.randn(E, generator=_gen(2), device="cuda")
    _check_logits(x, w, bias, tq.exl3_router_logits(x, tq.router(w, bias=bias)))


@pytest.mark.parametrize("T", [3, 200])
def test_logits_of_strided_rows_leave_the_rest_alone(T):
    """x is a slice of wider rows whose other columns are NaN; what lies past the logits stays."""
    wide = torch.full((T, 1024), math.nan, dtype=torch.float16, device="cuda")
    x, w = _inputs(T, 512, 40, False)
    wide[:, 256:768] = x
    buf = torch.full((T * 40 + 64,), 7.0, device="cuda")
    out = buf[:T * 40].view(T, 40)
    tq.exl3_router_logits(wide[:, 256:768], tq.router(w), logits=out)
    _check_logits(x, w, None, out)
    assert (buf[T * 40:] == 7).all()


@pytest.mark.parametrize("T", [4, 64])
def test_packed_weights_keep_22_bits(T):
    """Rows of x with a single 1: each logit is one weight, off by 2^-22 of it and by
    half a step of 2^-49 of its expert's largest."""
    E, k = 24, 64
    g = _gen(5)
    w = torch.randn((E, k), generator=g, device="cuda") * torch.exp(8 * torch.randn((E, k), generator=g, device="cuda"))
    w[3] *= 1e20
    w[4] *= 1e-20
    w[5] = 0
    x = torch.zeros((T, k), dtype=torch.float16, device="cuda")
    x[torch.arange(T), torch.arange(T) % k] = 1
    got = tq.exl3_router_logits(x, tq.router(w)).double()
    want = w.double().t()[torch.arange(T) % k]
    # (and the two roundings of the sum of the parts and of the power of two's product, none of which adds to a single
    # product: hi + 2^-11 lo has 22 bits)
    tol = want.abs() * 2.0 ** -22 + w.double().abs().amax(1)[None] * 2.0 ** -49
    assert ((got - want).abs() <= tol).all()


def test_rows_past_32_bits():
    """x and logits of more than 2^31 elements: the last rows."""
    k, E, tail = 17408, 8, 100
    x = torch.zeros((130000, k), dtype=torch.float16, device="cuda")
    xs, w = _inputs(tail, k, E, False)
    x[-tail:] = xs
    _check_logits(xs, w, None, tq.exl3_router_logits(x, tq.router(w))[-tail:])
    del x
    l = torch.zeros((2200000, 1024), dtype=torch.float16, device="cuda")
    l[-tail:] = _rand_logits(tail, 1024, seed=20, half=True)
    ids, got = tq.exl3_route(l, tq.route_rule(4))
    want_ids, want = _route_exact(l[-tail:], 4, "softmax", None, 1, 1, "max", True, 1.0)
    assert torch.equal(ids[-tail:].long(), want_ids) and torch.allclose(got[-tail:].double(), want, rtol=W_TOL)


def test_logits_repeat_bit_for_bit():
    x, w = _inputs(700, 2048, 256, True)
    r = tq.router(w)
    first = tq.exl3_router_logits(x, r)
    for _ in range(3):
        assert torch.equal(first, tq.exl3_router_logits(x, r))


# ------------------------------------------------------------------- routing

def _route_exact(l, topk, score, bias, groups, kept, group, renorm, scale):
    """The rule in 64 bits; NaN and barred experts as documented."""
    l = l.double()
    T, E = l.shape
    if score == "softmax":
        top = l.amax(-1, keepdim=True)
        e = (l - torch.where(top == -math.inf, 0.0, top)).exp()
        tot = e.sum(-1, keepdim=True)
        s = torch.where(tot == 0, 0.0, e / tot)
    else:
        s = torch.sigmoid(l)
    b = torch.zeros(E, dtype=torch.float64, device=l.device) if bias is None else bias.double()
    c = s + b
    if bias is None and (group == "max" or kept == groups):
        c = l                                                # both scores are monotone
    if kept < groups:
        v = c.view(T, groups, -1).sort(dim=-1, descending=True).values
        v = v[..., 0] if group == "max" or v.shape[-1] == 1 else v[..., 0] + v[..., 1]
        keep = v.sort(dim=-1, descending=True, stable=True).indices[:, :kept]
        mask = torch.zeros((T, groups), dtype=torch.bool, device=l.device).scatter_(1, keep, True)
        # left out ranks below barred
        c = torch.where(mask.repeat_interleave(E // groups, 1), c.clamp(min=-1e300), -math.inf)
    ids = c.sort(dim=-1, descending=True, stable=True).indices[:, :topk]
    if not renorm:
        return ids, torch.where(b[ids] == -math.inf, 0.0, s.gather(1, ids)) * scale
    # shares of the sum from the scores' logarithms: scores below 64 bits' range (a
    # row of the type's lowest value) have shares too
    z = (l if score == "softmax" else torch.nn.functional.logsigmoid(l)).gather(1, ids)
    z = torch.where(b[ids] == -math.inf, -math.inf, z)
    top = z.amax(-1, keepdim=True)
    e = (z - torch.where(top == -math.inf, 0.0, top)).exp()
    tot = e.sum(-1, keepdim=True)
    return ids, torch.where(tot == 0, 0.0, e / tot) * scale


# A weight: its exponential (2 units) of an argument off by a rounding of up to
# 40, sums of up to 32 + 5 terms over a row's 1024 or the chosen 32, a division,
# a product: below (2 + 40 + 37 + 3) 2^-24 < 2^-17.
W_TOL = 2.0 ** -17


def _check_route(l, topk, score="softmax", bias=None, groups=1, kept=None, group="max", renorm=True, scale=1.0):
    kept = groups if kept is None else kept
    rule = tq.route_rule(topk, score=tq.EXL3_SCORE_SOFTMAX if score == "softmax" else tq.EXL3_SCORE_SIGMOID, bias=bias,
                         groups=groups, groups_kept=kept,
                         group_score=tq.EXL3_GROUP_MAX if group == "max" else tq.EXL3_GROUP_TOP2, renormalise=renorm,
                         scale=scale)
    ids, w = tq.exl3_route(l, rule)
    want_ids, want_w = _route_exact(l, topk, score, bias, groups, kept, group, renorm, scale)
    assert torch.equal(ids.long(), want_ids)
    assert ((w.double() - want_w).abs() <= W_TOL * want_w.abs() + 1e-37).all()
    return ids, w


def _rand_logits(T, E, seed=0, half=False):
    l = 2 * torch.randn((T, E), generator=_gen(seed), device="cuda")
    return l.half() if half else l


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("score,renorm,biased", [("softmax", True, False), ("softmax", False, False),
                                                 ("sigmoid", True, False), ("sigmoid", False, True),
                                                 ("softmax", False, True), ("softmax", True, True)])
@pytest.mark.parametrize("T,E,topk", [(1, 256, 8), (333, 256, 8), (50, 60, 4), (50, 1, 1), (50, 8, 8), (50, 32, 32),
                                      (70, 33, 2), (40, 1024, 32), (40, 500, 6), (64, 128, 1)])
def test_route(T, E, topk, score, renorm, biased, half):
    bias = 0.1 * torch.randn(E, generator=_gen(9), device="cuda") if biased else None
    _check_route(_rand_logits(T, E, half=half), topk, score, bias, renorm=renorm, scale=1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group", ["max", "top2"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,groups,kept,topk", [(256, 8, 4, 8), (160, 8, 3, 6), (64, 32, 5, 10), (33, 3, 2, 4),
                                                (16, 16, 4, 4), (1024, 32, 1, 32), (60, 5, 1, 12), (96, 2, 1, 3)])
def test_route_groups(E, groups, kept, topk, biased, group, score):
    bias = 0.1 * torch.randn(E, generator=_gen(8), device="cuda") if biased else None
    _check_route(_rand_logits(200, E, seed=3), topk, score, bias, groups, kept, group)


@pytest.mark.parametrize("T", [1, 4097])
def test_many_rows_are_all_routed(T):
    _check_route(_rand_logits(T, 256, seed=4), 8, "sigmoid", 0.1 * torch.randn(256, generator=_gen(1), device="cuda"), 8, 4,
                 "top2")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_equal_values_go_to_the_lower_id(score, biased):
    """Logits of a few values only: ties everywhere, -0 and 0 among them."""
    l = torch.randint(-1, 2, (300, 64), generator=_gen(6), device="cuda").float()
    l[l == 0] *= torch.where(torch.rand(300, 64, generator=_gen(7), device="cuda") < 0.5, 1.0, -1.0)[l == 0]
    bias = torch.full((64,), 0.25, device="cuda") if biased else None
    _check_route(l, 8, score, bias)
    _check_route(l, 8, score, bias, groups=8, kept=3, group="top2")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_values_closer_than_fp32(score):
    """Experts whose scores differ by the bias' difference up to a few 1e-9: fp32
    does not tell s + b apart, 64 bits do."""
    T, E = 64, 64
    g = _gen(11)
    l = torch.randn((T, E), generator=g, device="cuda")
    one = l[:, :1].clone()
    l[:, ::2] = one                                       # the same score,
    bias = torch.zeros(E, device="cuda")
    bias[::2] = 1.0
    l[:, 0:16:2] += torch.linspace(0, 7, 8, device="cuda") * 2.0 ** -22     # then a few units apart
    _check_route(l, 8, score, bias)
    _check_route(l, 4, score, bias, groups=16, kept=5, group="top2")


@pytest.mark.parametrize("low", [-math.inf, torch.finfo(torch.float32).min])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_masked_logits(low, score, renorm, biased):
    """Rows with some, almost all and all experts masked."""
    l = _rand_logits(6, 40, seed=12)
    l[1, 10:] = low
    l[2, 3:] = low
    l[3, :] = low
    l[4, :-1] = low
    bias = 0.1 * torch.randn(40, generator=_gen(13), device="cuda") if biased else None
    ids, w = _check_route(l, 4, score, bias, renorm=renorm)
    assert all(len(set(r)) == 4 for r in ids.tolist()) and not w.isnan().any()
    if low == -math.inf:
        assert (w[3] == 0).all()


def test_sigmoid_weights_of_very_low_logits_keep_their_ratios():
    l = torch.full((1, 8), -300.0, device="cuda")
    l[0, 2], l[0, 5] = -200.0, -201.0
    ids, w = tq.exl3_route(l, tq.route_rule(2, score=tq.EXL3_SCORE_SIGMOID))
    assert ids.tolist() == [[2, 5]]
    e = math.exp(-1.0)
    assert torch.allclose(w.double().cpu(), torch.tensor([[1 / (1 + e), e / (1 + e)]], dtype=torch.float64), rtol=W_TOL)


def test_barred_experts():
    """A bias of -infinity: chosen only when nothing else is left, and then with weight 0."""
    l = _rand_logits(50, 16, seed=14)
    bias = torch.zeros(16, device="cuda")
    bias[3:] = -math.inf
    ids, w = _check_route(l, 5, "sigmoid", bias)
    assert (w[:, 3:] == 0).all() and ((ids[:, :3] < 3).all())
    _check_route(l, 5, "softmax", bias, groups=4, kept=2, group="top2")


def test_nan_stays_in_its_row():
    l = _rand_logits(4, 64, seed=15)
    clean = l.clone()
    l[1, 5] = math.nan
    l[2, :] = math.nan
    for rule in (tq.route_rule(4), tq.route_rule(4, renormalise=False), tq.route_rule(4, score=tq.EXL3_SCORE_SIGMOID),
                 tq.route_rule(4, bias=torch.zeros(64, device="cuda"), groups=8, groups_kept=2,
                               group_score=tq.EXL3_GROUP_TOP2)):
        ids, w = tq.exl3_route(l, rule)
        want_ids, want_w = tq.exl3_route(clean, rule)
        for r in (0, 3):
            assert torch.equal(ids[r], want_ids[r]) and torch.equal(w[r], want_w[r])
        assert all(len(set(r)) == 4 and 0 <= min(r) and max(r) < 64 for r in ids.tolist())
        assert w[2].isnan().all()


def test_route_of_strided_logits_writes_its_rows_only():
    wide = _rand_logits(20, 100, seed=16)
    ids = torch.full((21, 3), 77, dtype=torch.int32, device="cuda")
    w = torch.full((21, 3), 77.0, device="cuda")
    tq.exl3_route(wide[:, 7:60], tq.route_rule(3), ids=ids[:20], weights=w[:20])
    want_ids, want_w = _route_exact(wide[:, 7:60], 3, "softmax", None, 1, 1, "max", True, 1.0)
    assert torch.equal(ids[:20].long(), want_ids) and torch.allclose(w[:20].double(), want_w, rtol=W_TOL)
    assert (ids[20] == 77).all() and (w[20] == 77).all()


def test_empty_calls():
    assert tq.exl3_route(torch.empty((0, 8), device="cuda"), tq.route_rule(2))[0].shape == (0, 2)
    w = torch.zeros((8, 64), dtype=torch.float16, device="cuda")
    assert tq.exl3_router_logits(torch.empty((0, 64), dtype=torch.float16, device="cuda"), tq.router(w)).shape == (0, 8)


def test_a_rule_changed_after_it_was_made():
    """The rule's fields are read at the call: outputs are as wide as its topk then."""
    l = _rand_logits(30, 64, seed=17)
    rule = tq.route_rule(4)
    for topk in (4, 12, 2):
        rule.topk = topk
        ids, w = tq.exl3_route(l, rule)
        want_ids, want_w = tq.exl3_route(l, tq.route_rule(topk))
        assert ids.shape == (30, topk) and torch.equal(ids, want_ids) and torch.equal(w, want_w)
    rule.topk = 12
    with pytest.raises(ValueError, match="ids must be"):
        tq.exl3_route(l, rule, ids=torch.empty((30, 4), dtype=torch.int32, device="cuda"))
    rule.scale = 2.5
    assert torch.equal(tq.exl3_route(l, rule)[1], tq.exl3_route(l, tq.route_rule(12, scale=2.5))[1])


def test_sizes_of_a_router_stay():
    x, w = _inputs(3, 64, 16, False)
    r = tq.router(w)
    for name in ("E", "k"):
        with pytest.raises(AttributeError, match="size"):
            setattr(r, name, 128)
    _check_logits(x, w, None, tq.exl3_router_logits(x, r))


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("T,k,E", [(1, 256, 24), (8, 256, 24), (9, 256, 24), (64, 2048, 256), (300, 1048, 60), (4096, 512, 256)])
def test_infinities_in_x(T, k, E, fp32):
    """+-infinity times a weight's sign, NaN for a weight of zero or infinities that meet; other rows as they were."""
    x, w = _inputs(T, k, E, fp32, seed=21)
    w = torch.where(w.abs() < 2.0 ** -14, torch.full_like(w, 2.0 ** -14), w)     # (none that packing takes for zero)
    w[3, 5], w[E - 1, k - 1] = 0, 0
    w[7, 9] = 2.0 ** -10                                   # (of a low part of zero)
    r = tq.router(w)
    clean = tq.exl3_router_logits(x, r)
    rows = sorted({0, T // 2, T - 1})
    x[0, 5] = math.inf
    x[T // 2, 9] = -math.inf
    x[T - 1, k - 1], x[T - 1, k // 2] = math.inf, math.inf
    got = tq.exl3_router_logits(x, r)
    want = (x[rows].double()[:, None] * w.double()).sum(-1)
    assert torch.equal(got[rows].isnan(), want.isnan()) and not want.isfinite().any()
    inf = want.isinf()
    assert inf.any() and want.isnan().any() and torch.equal(got[rows][inf].double(), want[inf])
    rest = [t for t in range(T) if t not in rows]
    assert torch.equal(got[rest], clean[rest])


@pytest.mark.parametrize("T", [3, 40])
def test_rows_of_weights_that_are_not_finite(T):
    """NaN for their expert, nothing for the others, whatever the number of rows."""
    x, w = _inputs(T, 256, 24, True, seed=22)
    clean = tq.exl3_router_logits(x, tq.router(w))
    w[4, 10], w[9, 200], w[20, 0] = math.inf, math.nan, -math.inf
    got = tq.exl3_router_logits(x, tq.router(w))
    bad = [4, 9, 20]
    rest = [e for e in range(24) if e not in bad]
    assert got[:, bad].isnan().all() and torch.equal(got[:, rest], clean[:, rest])
