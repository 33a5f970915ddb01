"""GPU parity of exl3_qk_norm_rope and exl3_qkv_append against the plain 64-bit
form; bounds are derived in tests/attention_ref.py."""
import math

import pytest
import torch

import trellis_quantized_gb300 as tq
from attention_ref import assert_transform, transform

pytestmark = pytest.mark.gpu


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _make(T, Hq, Hkv, D, R, norm, dtype, g, spread=3.0):
    q = (spread * torch.randn((T, Hq, D), generator=g, device="cuda")).to(dtype)
    k = (spread * torch.randn((T, Hkv, D), generator=g, device="cuda")).to(dtype)
    v = (spread * torch.randn((T, Hkv, D), generator=g, device="cuda")).to(dtype)
    qn = kn = None
    if norm in ("both", "q"):
        qn = (1 + 0.5 * torch.randn(D, generator=g, device="cuda")).half()
    if norm in ("both", "k"):
        kn = (1 + 0.5 * torch.randn(D, generator=g, device="cuda")).half()
    f = None if R == 0 else tq.exl3_rope_frequencies(R)[0].cuda()
    return q, k, v, qn, kn, f


@pytest.mark.parametrize("D,R", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 2), (256, 64), (256, 256), (128, 20),
                                 (64, 36), (256, 250), (128, 0)])
@pytest.mark.parametrize("layout", [tq.EXL3_ROPE_HALF, tq.EXL3_ROPE_PAIRS])
@pytest.mark.parametrize("norm", ["both", "none"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_transform(D, R, layout, norm, dtype):
    T, Hq, Hkv = 13, 5, 3
    q, k, _, qn, kn, f = _make(T, Hq, Hkv, D, R, norm, dtype, _gen(D + R + layout))
    pos = _i32([0, 1, 2, 7, 100, 4095, 65535, 999983, 2 ** 24 + 1, 2 ** 31 - 1, -1, -70000, 31])
    mag = 1.25
    ht = tq.head_transform(qn, kn, 1e-6, f, layout, mag)
    for od in (tq.EXL3_OUT_F16, tq.EXL3_OUT_F32):
        qo, ko = tq.exl3_qk_norm_rope(q, k, pos if R else None, ht, out_dtype=od)
        for x, w, y, what in ((q, qn, qo, "q"), (k, kn, ko, "k")):
            want, size = transform(x, w, 1e-6, pos, f, layout == tq.EXL3_ROPE_PAIRS, mag)
            assert_transform(y, want, size, what)


@pytest.mark.parametrize("T", [1, 2, 31, 700])
@pytest.mark.parametrize("Hq,Hkv,D", [(40, 8, 128), (16, 2, 256), (1, 1, 64), (33, 0, 64), (65, 5, 256)])
@pytest.mark.parametrize("norm", ["q", "k"])
def test_head_counts(T, Hq, Hkv, D, norm):
    q, k, _, qn, kn, f = _make(T, Hq, max(Hkv, 1), D, D, norm, torch.float16, _gen(T + Hq))
    k = k if Hkv else None
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 37
    qo, ko = tq.exl3_qk_norm_rope(q, k, pos, tq.head_transform(qn, kn, 1e-5, f))
    assert_transform(qo, *transform(q, qn, 1e-5, pos, f, False, 1.0), "q")
    if Hkv:
        assert_transform(ko, *transform(k, kn, 1e-5, pos, f, False, 1.0), "k")
    else:
        assert ko is None


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("R", [128, 20])
def test_in_place_and_strided(dtype, R):
    """q and k as slices of one [T, n] projection, and the output over the input."""
    T, Hq, Hkv, D = 50, 6, 2, 128
    g = _gen(3)
    wide = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device="cuda").to(dtype)
    q = wide[:, :Hq * D].unflatten(1, (Hq, D))
    k = wide[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    _, _, _, qn, kn, f = _make(1, 1, 1, D, R, "both", dtype, g)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    ht = tq.head_transform(qn, kn, 1e-6, f)
    od = tq.EXL3_OUT_F32 if dtype == torch.float32 else tq.EXL3_OUT_F16
    qo, ko = tq.exl3_qk_norm_rope(q, k, pos, ht, out_dtype=od)
    assert_transform(qo, *transform(q, qn, 1e-6, pos, f, False, 1.0), "strided q")
    qc, kc = q.contiguous(), k.contiguous()
    tq.exl3_qk_norm_rope(qc, kc, pos, ht, q_out=qc, k_out=kc, out_dtype=od)
    assert torch.equal(qc, qo) and torch.equal(kc, ko)


def test_zero_rows_and_large_values():
    """A zero head stays zero (eps), fp32 inputs past fp16's range come back normed."""
    T, D = 4, 128
    q = torch.randn((T, 2, D), device="cuda") * 1e6
    q[1] = 0
    w = torch.ones(D, dtype=torch.float16, device="cuda")
    f = tq.exl3_rope_frequencies(D)[0].cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    y, _ = tq.exl3_qk_norm_rope(q, None, pos, tq.head_transform(w, None, 1e-6, f))
    assert not y[1].any()
    assert_transform(y, *transform(q, w, 1e-6, pos, f, False, 1.0))


def _cache(pages, page, Hkv, D, order, g):
    shape = (pages, page, Hkv, D) if order == "tokens" else (pages, Hkv, page, D)
    both = torch.randn((2,) + shape, generator=g, device="cuda").half()
    k, v = both[0], both[1]
    return (k, v) if order == "tokens" else (k.transpose(1, 2), v.transpose(1, 2))


def _append(new, old, Hq, Hkv, D, R, page, order, dtype, layout=tq.EXL3_ROPE_HALF, norm="both", pad=0, positions=None,
            seed=0):
    g = _gen(seed + sum(new) * 13 + D)
    T = sum(new) + pad
    q, k, v, qn, kn, f = _make(T, Hq, Hkv, D, R, norm, dtype, g)
    need = [(n + o + page - 1) // page for n, o in zip(new, old)]
    kc, vc = _cache(sum(need) + 2, page, Hkv, D, order, g)
    perm = torch.randperm(sum(need) + 2, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(new), max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at, starts, pos, places = 0, [0], [], []
    for b, (n, o) in enumerate(zip(new, old)):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        starts.append(starts[-1] + n)
        p = torch.arange(o, o + n, device="cuda")
        pos.append(p)
        places.append((table[b].long()[p // page], p % page))
    pos = torch.cat(pos)
    before_k, before_v = kc.clone(), vc.clone()
    ht = tq.head_transform(qn, kn, 1e-6, f, layout)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    batch = tq.paged_batch(_i32(starts), _i32([n + o for n, o in zip(new, old)]), table)
    qo = tq.exl3_qkv_append(q, k, v, batch, tq.kv_cache(kc, vc), ht, positions=positions, workspace_buf=ws)
    assert tq.exl3_check_device_error(ws) == 0
    n = sum(new)
    at_pos = pos if positions is None else positions[:n]
    pg, off = torch.cat([p for p, _ in places]), torch.cat([o for _, o in places])
    pairs = layout == tq.EXL3_ROPE_PAIRS
    assert_transform(qo[:n], *transform(q[:n], qn, 1e-6, at_pos, f, pairs, 1.0), "q")
    assert not qo[n:].any()
    assert_transform(kc[pg, off], *transform(k[:n], kn, 1e-6, at_pos, f, pairs, 1.0), "k")
    assert torch.equal(vc[pg, off], v[:n].half())
    before_k[pg, off], before_v[pg, off] = kc[pg, off], vc[pg, off]
    assert torch.equal(before_k, kc) and torch.equal(before_v, vc), "other places are untouched"


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("page,order", [(16, "tokens"), (48, "heads"), (256, "tokens")])
@pytest.mark.parametrize("Hq,Hkv,D,R", [(40, 8, 128, 128), (16, 2, 256, 64), (24, 8, 64, 20)])
@pytest.mark.parametrize("new,old", [([1], [0]), ([1, 1, 1], [15, 16, 1000]), ([100, 1, 0, 33], [0, 47, 5, 300])])
def test_append(dtype, page, order, Hq, Hkv, D, R, new, old):
    _append(new, old, Hq, Hkv, D, R, page, order, dtype)


def test_append_many_sequences():
    old = [(7 * i) % 97 for i in range(1500)]
    new = [1 + (i % 3 == 0) for i in range(1500)]
    _append(new, old, 8, 2, 64, 64, 16, "tokens", torch.float16, layout=tq.EXL3_ROPE_PAIRS)


def test_append_padding_rows_and_positions():
    _append([3, 2], [10, 0], 8, 2, 128, 128, 16, "tokens", torch.float16, pad=4)
    pos = _i32([5, 5, 900000, -3, 2, 0, 0])
    _append([3, 2], [10, 0], 8, 2, 128, 128, 16, "tokens", torch.float16, pad=2, positions=pos, norm="none")


def test_append_bad_pages_are_reported_and_skipped():
    g = _gen(1)
    q, k, v, qn, kn, f = _make(2, 8, 2, 128, 128, "both", torch.float16, g)
    kc, vc = _cache(4, 16, 2, 128, "tokens", g)
    k0, v0 = kc.clone(), vc.clone()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    ht, cache = tq.head_transform(qn, kn, 1e-6, f), tq.kv_cache(kc, vc)
    for lens, table in (([40], [[0, 1, -1]]), ([40], [[0, 1, 4]]), ([60], [[0, 1, 2]]), ([0], [[0, 1, 2]])):
        tq.exl3_qkv_append(q, k, v, tq.paged_batch(_i32([0, 2]), _i32(lens), _i32(table)), cache, ht, workspace_buf=ws)
        assert tq.exl3_check_device_error(ws) != 0
        assert torch.equal(kc, k0) and torch.equal(vc, v0)


def test_append_in_a_graph_on_another_stream():
    g = _gen(9)
    q, k, v, qn, kn, f = _make(2, 8, 2, 128, 128, "both", torch.float16, g)
    kc, vc = _cache(4, 16, 2, 128, "tokens", g)
    lens = _i32([5, 9])
    batch = tq.paged_batch(_i32([0, 1, 2]), lens, _i32([[0], [3]]))
    ht, cache = tq.head_transform(qn, kn, 1e-6, f), tq.kv_cache(kc, vc)
    qo = torch.empty_like(q)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        tq.exl3_qkv_append(q, k, v, batch, cache, ht, q_out=qo, workspace_buf=ws)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.exl3_qkv_append(q, k, v, batch, cache, ht, q_out=qo, workspace_buf=ws)
    for a, b in ((1, 1), (16, 2), (7, 16)):
        lens.copy_(_i32([a, b]))
        graph.replay()
        torch.cuda.synchronize()
        pos = _i32([a - 1, b - 1])
        assert_transform(qo, *transform(q, qn, 1e-6, pos, f, False, 1.0), "q")
        got = torch.stack([kc[0, a - 1], kc[3, b - 1]])
        assert_transform(got, *transform(k, kn, 1e-6, pos, f, False, 1.0), "k")
        assert torch.equal(torch.stack([vc[0, a - 1], vc[3, b - 1]]), v)


def test_append_past_two_gigabytes():
    page, Hkv, D = 256, 8, 256
    pages = (2 ** 31 + 2 ** 26) // (page * Hkv * D) + 1
    kc = torch.zeros((pages, page, Hkv, D), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    q, k, v, qn, kn, f = _make(3, 8, Hkv, D, D, "both", torch.float16, _gen(2))
    batch = tq.paged_batch(_i32([0, 3]), _i32([10]), _i32([[pages - 1]]))
    tq.exl3_qkv_append(q, k, v, batch, tq.kv_cache(kc, vc), tq.head_transform(qn, kn, 1e-6, f))
    pos = _i32([7, 8, 9])
    assert_transform(kc[pages - 1, 7:10], *transform(k, kn, 1e-6, pos, f, False, 1.0), "k")
    assert torch.equal(vc[pages - 1, 7:10], v)
    assert math.isclose(float(kc[:pages - 1].abs().max()), 0.0)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("Hq,Hkv,D,R", [(4, 4, 64, 64), (5, 3, 64, 20), (6, 1, 128, 128)])
def test_append_more_tokens_than_warps(Hq, Hkv, D, R, dtype):
    """Every warp goes through several tokens, and through the ends of sequences and pages."""
    _append([1, 4001, 0, 5003, 17, 2], [30, 0, 9, 77, 15, 0], Hq, Hkv, D, R, 16, "tokens", dtype, pad=1100)


def test_transform_of_more_tokens_than_warps():
    T = 9001
    q, k, _, qn, kn, f = _make(T, 5, 3, 64, 64, "both", torch.float16, _gen(4))
    pos = torch.randint(-100, 1 << 20, (T,), generator=_gen(5), device="cuda", dtype=torch.int32)
    qo, ko = tq.exl3_qk_norm_rope(q, k, pos, tq.head_transform(qn, kn, 1e-6, f))
    assert_transform(qo, *transform(q, qn, 1e-6, pos, f, False, 1.0), "q")
    assert_transform(ko, *transform(k, kn, 1e-6, pos, f, False, 1.0), "k")


def test_append_rows_before_the_first_sequence():
    first, new, page, D = 5002, 4500, 16, 64
    T = first + new + 3
    g = _gen(8)
    q, k, v, qn, kn, f = _make(T, 4, 4, D, D, "both", torch.float16, g)
    pages = (new + 40 + page - 1) // page
    kc, vc = _cache(pages, page, 4, D, "tokens", g)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    # the first sequence has no rows
    batch = tq.paged_batch(_i32([first, first, first + new]), _i32([3, new + 40]), torch.stack([table.flip(0), table]))
    qo = tq.exl3_qkv_append(q, k, v, batch, tq.kv_cache(kc, vc), tq.head_transform(qn, kn, 1e-6, f), workspace_buf=ws)
    assert tq.exl3_check_device_error(ws) == 0
    mine = slice(first, first + new)
    pos = torch.arange(40, 40 + new, device="cuda")
    assert not qo[:first].any() and not qo[first + new:].any()
    assert_transform(qo[mine], *transform(q[mine], qn, 1e-6, pos, f, False, 1.0), "q")
    pg, off = table.long()[pos // page], pos % page
    assert_transform(kc[pg, off], *transform(k[mine], kn, 1e-6, pos, f, False, 1.0), "k")
    assert torch.equal(vc[pg, off], v[mine])


def test_append_with_a_length_below_its_new_tokens():
    """The tokens without a place are reported, the others are where they belong."""
    new, n, page, D = 6000, 4000, 16, 64
    g = _gen(12)
    q, k, v, qn, kn, f = _make(new, 4, 4, D, D, "both", torch.float16, g)
    kc, vc = _cache(n // page, page, 4, D, "tokens", g)
    table = torch.randperm(n // page, generator=g, device="cuda").to(torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    batch = tq.paged_batch(_i32([0, new]), _i32([n]), table[None].contiguous())
    qo = tq.exl3_qkv_append(q, k, v, batch, tq.kv_cache(kc, vc), tq.head_transform(qn, kn, 1e-6, f), workspace_buf=ws)
    assert tq.exl3_check_device_error(ws) != 0
    pos = torch.arange(n, device="cuda")
    pg, off = table.long()[pos // page], pos % page
    assert not qo[:new - n].any()
    assert_transform(qo[new - n:], *transform(q[new - n:], qn, 1e-6, pos, f, False, 1.0), "q")
    assert_transform(kc[pg, off], *transform(k[new - n:], kn, 1e-6, pos, f, False, 1.0), "k")
    assert torch.equal(vc[pg, off], v[new - n:])
