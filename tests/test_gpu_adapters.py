"""exl3_adapter_plan and exl3_adapter_add against their definition in 64 bits."""
import math

import pytest
import torch

import trellis_quantized_gb300 as tq

pytestmark = pytest.mark.gpu


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pool(N, R, k, n, ranks=None, seed=0, junk=0.0):
    """Adapters; past a rank lies `junk` in A and in B from the next multiple of 16 on, 9 before it."""
    g = _gen(seed)
    a = (torch.randn((N, R, k), generator=g, device="cuda") / math.sqrt(k)).half()
    b = (torch.randn((N, n, R), generator=g, device="cuda") / math.sqrt(R)).half()
    scale = torch.rand(N, generator=g, device="cuda") + 0.5
    for i, r in enumerate(ranks or []):
        a[i, r:] = junk
        b[i, :, r:] = 9.0
        b[i, :, (r + 15) // 16 * 16:] = junk
    rank = None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device="cuda")
    return a, b, scale, rank


def _large(T, R, n):
    """Calls on tiles of 128 rows (the library's rule; smaller ones run on tiles of 16)."""
    return T >= 48 and T * (R + 16) ** 2 * n >= 1 << 34


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(rows, first=0):
    out = [first]
    for r in rows:
        out.append(out[-1] + r)
    return out


def _reference(x, y, pool, rows, ids, first=0):
    """out in 64 bits and a bound on what the kernels may be off by, before the output's own rounding.

    h is a sum of k exact products in fp32 (k units of sum |x a|), enters the
    second product with 22 bits (2^-22 of the row's largest at most), which has
    2 R terms and as many roundings; one more each for the scale and the sum."""
    a, b, scale, rank = pool
    R, k = a.shape[1], a.shape[2]
    want, tol = y.double().clone(), torch.zeros(y.shape, dtype=torch.float64, device="cuda")
    t = first
    for n, i in zip(rows, ids):
        if i >= 0 and n:
            r = R if rank is None else int(rank[i])
            A, B, s = a[i, :r].double(), b[i, :, :r].double(), float(scale[i])
            xd = x[t:t + n].double()
            h, size = xd @ A.t(), xd.abs() @ A.abs().t()
            err = size * (k * 2.0 ** -23) + h.abs().amax(1, keepdim=True) * 2.0 ** -22 if r else size
            d = s * (h @ B.t())
            bound = s * ((err + h.abs() * (2 * R + 2) * 2.0 ** -23) @ B.abs().t())
            want[t:t + n] += d
            tol[t:t + n] = bound + want[t:t + n].abs() * 2.0 ** -24
        t += n
    return want, tol


def _check(out, want, tol):
    assert torch.isfinite(out).all()
    half_step = torch.finfo(out.dtype).eps / 2 if out.dtype == torch.float16 else 0.0
    # fp16 below its normal range: half of its smallest step
    tol = tol + (want.abs() + tol) * half_step + (2.0 ** -25 if out.dtype == torch.float16 else 0.0)
    off = (out.double() - want).abs() - tol
    assert (off <= 0).all(), f"{int((off > 0).sum())} off, by up to {float(off.max())}"


def _run(rows, ids, N, R, k, n, fp32=False, ranks=None, in_place=False, seed=0, junk=0.0):
    T = sum(rows)
    g = _gen(seed + 100)
    x = torch.randn((T, k), generator=g, device="cuda").half()
    y = torch.randn((T, n), generator=g, device="cuda").to(torch.float32 if fp32 else torch.float16)
    pool = _pool(N, R, k, n, ranks, seed, junk)
    plan = tq.exl3_adapter_plan(_i32(_starts(rows)), _i32(ids), T, N)
    want, tol = _reference(x, y, pool, rows, ids)
    out = y if in_place else torch.full_like(y, math.nan)
    ws = torch.zeros(tq.exl3_adapter_add_workspace_size(T, R), dtype=torch.uint8, device="cuda")
    tq.exl3_adapter_add(x, y, tq.adapters(*pool), plan, out=out, workspace_buf=ws)
    assert tq.exl3_check_device_error(plan.data) == 0 and tq.exl3_check_device_error(ws) == 0
    _check(out, want, tol)
    return out


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("R", [8, 16, 24, 32, 64, 104, 128])
@pytest.mark.parametrize("k,n", [(128, 128), (1024, 640), (5120, 512)])
def test_one_row(R, k, n, fp32):
    _run([1], [1], 3, R, k, n, fp32)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("rows", [[16], [17], [1, 3, 15, 1], [1] * 40, [5, 0, 30, 1, 1, 2], [128], [129, 1], [100, 300]])
def test_ragged_sequences(rows, fp32, in_place):
    ids = [(3 * i + 1) % 5 for i in range(len(rows))]
    _run(rows, ids, 5, 16, 512, 384, fp32, in_place=in_place)


@pytest.mark.parametrize("R", [8, 16, 40, 64, 128])
@pytest.mark.parametrize("rows", [[600], [200, 333, 1, 1, 1, 90], [127, 128, 129, 255, 257]])
@pytest.mark.parametrize("fp32", [False, True])
def test_prompts(rows, R, fp32):
    _run(rows, [i % 3 for i in range(len(rows))], 3, R, 1024, 1152, fp32)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("R,k,n", [(8, 128, 76800), (16, 17408, 43008), (24, 19200, 27008), (40, 512, 13696),
                                   (64, 256, 8320), (72, 8192, 5632), (128, 4096, 2176), (128, 128, 5120)])
@pytest.mark.parametrize("rows", [[600], [200, 333, 1, 1, 1, 90], [127, 128, 129, 255, 1, 0, 11, 12, 13, 50]])
def test_large_tiles(rows, R, k, n, fp32, in_place):
    assert _large(sum(rows), R, n)
    _run(rows, [i % 3 for i in range(len(rows))], 3, R, k, n, fp32, in_place=in_place)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("R,k,n", [(128, 384, 128), (104, 640, 256)])
def test_large_tiles_of_few_columns(R, k, n, fp32):
    rows = [9000, 1, 0, 900, 30]
    assert _large(sum(rows), R, n)
    _run(rows, [0, 1, 2, 1, -1], 3, R, k, n, fp32)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("rows", [[4000], [1, 2100, 7, 900, 16, 17]])
def test_many_small_tiles(rows, fp32):
    """Prompts of a small rank: hundreds of tiles of 16 rows, in clusters of two."""
    assert not _large(sum(rows), 16, 1280)
    _run(rows, [i % 3 for i in range(len(rows))], 3, 16, 1024, 1280, fp32)


@pytest.mark.parametrize("fp32", [False, True])
def test_large_tiles_of_scattered_rows(fp32):
    """Sequences of one to five rows of five adapters and none: every tile gathers."""
    rows = [1 + i % 5 for i in range(300)]
    ids = [(i * 7) % 6 - 1 for i in range(300)]
    assert _large(sum(rows), 64, 4608)
    _run(rows, ids, 5, 64, 512, 4608, fp32)
    _run(rows, ids, 5, 64, 512, 4608, fp32, in_place=True)


@pytest.mark.parametrize("rows,R,n", [([1] * 30, 32, 256), ([400, 1, 30, 200], 32, 256), ([400, 1, 30, 200], 64, 8192)])
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_without_an_adapter_keep_y(rows, R, n, fp32, in_place):
    ids = [-1 if i % 3 else 2 for i in range(len(rows))]
    assert _large(sum(rows), R, n) == (n > 256)
    _run(rows, ids, 4, R, 256, n, fp32, in_place=in_place)
    _run(rows, [-1] * len(rows), 4, R, 256, n, fp32, in_place=in_place)


@pytest.mark.parametrize("rows,n", [([1, 1, 2, 1, 1, 1], 512), ([300, 1, 5, 140, 200, 131], 512),
                                    ([300, 1, 5, 140, 200, 131], 8192)])
@pytest.mark.parametrize("R,ranks", [(64, [8, 64, 16, 33, 0, 40]), (128, [128, 1, 64, 65, 100, 16])])
def test_ranks_and_what_lies_past_them(rows, n, R, ranks):
    """NaN past an adapter's rank in A, and in B past the next multiple of 16."""
    assert _large(sum(rows), R, n) == (n > 512)
    _run(rows, list(range(6)), 6, R, 512, n, True, ranks, junk=math.nan)


@pytest.mark.parametrize("rows,R,n", [([1] * 8, 16, 256), ([150, 20], 16, 256), ([150, 20], 128, 12288)])
def test_rows_outside_the_sequences_are_left_alone(rows, R, n):
    T, k = sum(rows) + 12, 256
    assert _large(T, R, n) == (n > 256)
    x = torch.randn((T, k), generator=_gen(1), device="cuda").half()
    y = torch.randn((T, n), generator=_gen(2), device="cuda").half()
    x[:5], x[-7:] = math.nan, math.nan
    pool = _pool(2, R, k, n)
    ids = [i % 2 for i in range(len(rows))]
    plan = tq.exl3_adapter_plan(_i32(_starts(rows, 5)), _i32(ids), T, 2)
    out = torch.full_like(y, 7.0)
    tq.exl3_adapter_add(x, y, tq.adapters(*pool), plan, out=out)
    want, tol = _reference(x, y, pool, rows, ids, 5)
    _check(out[5:-7], want[5:-7], tol[5:-7])
    assert (out[:5] == 7).all() and (out[-7:] == 7).all()


@pytest.mark.parametrize("rows,R,n", [([2, 1], 24, 384), ([180, 70], 24, 384), ([180, 70], 128, 8448)])
def test_strided_rows(rows, R, n):
    T, k = sum(rows), 256
    assert _large(T, R, n) == (n > 384)
    wx = torch.full((T, k + 64), math.nan, dtype=torch.float16, device="cuda")
    wy = torch.full((T, 2 * n), math.nan, dtype=torch.float32, device="cuda")
    wo = torch.full((T, n + 32), 7.0, dtype=torch.float32, device="cuda")
    x = torch.randn((T, k), generator=_gen(1), device="cuda").half()
    y = torch.randn((T, n), generator=_gen(2), device="cuda")
    wx[:, 64:], wy[:, n:] = x, y
    pool = _pool(2, R, k, n)
    plan = tq.exl3_adapter_plan(_i32(_starts(rows)), _i32([1, 0]), T, 2)
    tq.exl3_adapter_add(wx[:, 64:], wy[:, n:], tq.adapters(*pool), plan, out=wo[:, 16:n + 16])
    _check(wo[:, 16:n + 16].contiguous(), *_reference(x, y, pool, rows, [1, 0]))
    assert (wo[:, :16] == 7).all() and (wo[:, n + 16:] == 7).all()


@pytest.mark.parametrize("fp32", [False, True])
def test_out_on_16_bytes(fp32):
    """Large tiles whose output rows start on 16 bytes, not on 32."""
    T, R, k, n = 250, 128, 256, 8448
    assert _large(T, R, n)
    at = 4 if fp32 else 8
    x = torch.randn((T, k), generator=_gen(1), device="cuda").half()
    y = torch.randn((T, n), generator=_gen(2), device="cuda").to(torch.float32 if fp32 else torch.float16)
    wide = torch.full((T, n + 2 * at), 7.0, dtype=y.dtype, device="cuda")
    pool = _pool(2, R, k, n)
    plan = tq.exl3_adapter_plan(_i32([0, 33, T]), _i32([1, 0]), T, 2)
    tq.exl3_adapter_add(x, y, tq.adapters(*pool), plan, out=wide[:, at:n + at])
    _check(wide[:, at:n + at].contiguous(), *_reference(x, y, pool, [33, T - 33], [1, 0]))
    assert (wide[:, :at] == 7).all() and (wide[:, n + at:] == 7).all()


@pytest.mark.parametrize("T,R,k,n,N", [(130000, 8, 128, 17408, 2), (130000, 8, 17408, 128, 2),
                                       (130000, 64, 17408, 128, 2), (2, 128, 128, 17408, 1000),
                                       (200, 128, 128, 17408, 1000)])
def test_offsets_past_32_bits(T, R, k, n, N):
    """x, y and out, or a pool, of more than 2^31 elements: the last rows and the last adapter."""
    assert max(T * k, T * n, N * R * n) > 1 << 31
    tail = min(T, 70)
    x = torch.zeros((T, k), dtype=torch.float16, device="cuda")
    y = torch.zeros((T, n), dtype=torch.float16, device="cuda")
    x[-tail:] = torch.randn((tail, k), generator=_gen(1), device="cuda").half()
    y[-tail:] = torch.randn((tail, n), generator=_gen(2), device="cuda").half()
    a = torch.zeros((N, R, k), dtype=torch.float16, device="cuda")
    b = torch.zeros((N, n, R), dtype=torch.float16, device="cuda")
    small = _pool(1, R, k, n)
    a[-1], b[-1] = small[0][0], small[1][0]
    scale = torch.zeros(N, device="cuda")
    scale[-1] = small[2][0]
    out = torch.empty_like(y)
    plan = tq.exl3_adapter_plan(_i32([0, T - tail, T]), _i32([-1 if T == tail else 0, N - 1]), T, N)
    tq.exl3_adapter_add(x, y, tq.adapters(a, b, scale), plan, out=out)
    _check(out[-tail:], *_reference(x[-tail:], y[-tail:], small, [tail], [0]))
    if T > tail:
        assert (out[:T - tail:1009] == 0).all()


@pytest.mark.parametrize("size", [1e-6, 300.0])
@pytest.mark.parametrize("rows,R,n", [([3, 2], 16, 256), ([200, 60], 16, 256), ([200, 60], 128, 8192)])
def test_h_outside_fp16(rows, R, n, size):
    """x A^T of 1e-9 or of 1e6: its two parts are scaled by a power of two per row."""
    T, k = sum(rows), 512
    assert _large(T, R, n) == (n > 256)
    x = (torch.randn((T, k), generator=_gen(1), device="cuda") * size).half()
    y = torch.zeros((T, n), device="cuda")
    a, b, scale, rank = _pool(2, R, k, n)
    a = (a.float() * (300.0 if size > 1 else 0.01)).half()
    pool = (a, b, scale, rank)
    plan = tq.exl3_adapter_plan(_i32(_starts(rows)), _i32([0, 1]), T, 2)
    tq.exl3_adapter_add(x, y, tq.adapters(*pool), plan)
    _check(y, *_reference(x, torch.zeros_like(y), pool, rows, [0, 1]))


def test_a_row_does_not_depend_on_the_others():
    """Infinities and NaN in one row of a tile stay there."""
    for T, R, n in ((9, 16, 256), (140, 16, 256), (140, 128, 16384)):
        assert _large(T, R, n) == (n > 256)
        x = torch.randn((T, 256), generator=_gen(1), device="cuda").half()
        y = torch.randn((T, n), generator=_gen(2), device="cuda")
        pool = tq.adapters(*_pool(1, R, 256, n))
        plan = tq.exl3_adapter_plan(_i32([0, T]), _i32([0]), T, 1)
        clean = tq.exl3_adapter_add(x, y, pool, plan, out=torch.empty_like(y))
        x[3], x[5, 7] = math.nan, math.inf
        got = tq.exl3_adapter_add(x, y, pool, plan, out=torch.empty_like(y))
        keep = [t for t in range(T) if t not in (3, 5)]
        assert torch.equal(got[keep], clean[keep]) and got[3].isnan().all()


def test_bad_adapters_and_starts_are_recorded():
    T, k, n = 6, 128, 128
    x = torch.randn((T, k), generator=_gen(1), device="cuda").half()
    y = torch.randn((T, n), generator=_gen(2), device="cuda")
    pool = _pool(2, 8, k, n)
    for ids in ([0, 2, 1], [0, -2, 1]):                    # treated as none
        plan = tq.exl3_adapter_plan(_i32([0, 2, 4, 6]), _i32(ids), T, 2)
        out = tq.exl3_adapter_add(x, y, tq.adapters(*pool), plan, out=torch.zeros_like(y))
        assert tq.exl3_check_device_error(plan.data) != 0
        assert tq.exl3_check_device_error(plan.data) == 0
        _check(out, *_reference(x, y, pool, [2, 2, 2], [0, -1, 1]))
    for starts in ([0, 4, 2, 6], [-1, 2, 4, 6], [0, 2, 4, 7]):
        plan = tq.exl3_adapter_plan(_i32(starts), _i32([0, 1, 1]), T, 2, plan=plan)
        assert tq.exl3_check_device_error(plan.data) != 0
        out = tq.exl3_adapter_add(x, y, tq.adapters(*pool), plan, out=torch.full_like(y, 7.0))
        assert (out == 7).all()
    # a plan that was never filled
    empty = tq.AdapterPlan(T, 3, 2, x.device)
    ws = torch.zeros(tq.exl3_adapter_add_workspace_size(T, 8), dtype=torch.uint8, device="cuda")
    out = tq.exl3_adapter_add(x, y, tq.adapters(*pool), empty, out=torch.full_like(y, 7.0), workspace_buf=ws)
    assert (out == 7).all() and tq.exl3_check_device_error(ws) != 0


def test_many_adapters_and_sequences():
    """Every row its own adapter out of 3000, and 3000 sequences of one."""
    rows = [1] * 3000
    _run(rows, [(7 * i) % 3000 for i in range(3000)], 3000, 8, 128, 128)
    _run(rows, [1] * 3000, 2, 8, 128, 128)
    assert _large(3000, 8, 14976)
    _run(rows, [(7 * i) % 3000 for i in range(3000)], 3000, 8, 128, 14976)
    _run(rows, [1] * 3000, 2, 8, 128, 14976)


@pytest.mark.parametrize("rows,R,n", [([1] * 50, 16, 512), ([3, 1, 1, 30, 2, 9] * 7, 24, 256), ([1, 200, 3, 70, 1, 1], 128, 8192)])
def test_the_same_call_gives_the_same_bits(rows, R, n):
    """Plans made again, for sequences whose rows fall into tiles of different sizes."""
    T, k = sum(rows), 512
    x = torch.randn((T, k), generator=_gen(1), device="cuda").half()
    y = torch.randn((T, n), generator=_gen(2), device="cuda")
    ad, q, ids = tq.adapters(*_pool(2, R, k, n)), _i32(_starts(rows)), _i32([i % 2 for i in range(len(rows))])
    first = None
    for _ in range(8):
        plan = tq.exl3_adapter_plan(q, ids, T, 2)
        out = tq.exl3_adapter_add(x, y, ad, plan, out=torch.empty_like(y))
        first = out if first is None else first
        assert torch.equal(out, first)


def test_more_sequences_than_threads():
    """2500 sequences of zero to three rows: places counted in several stretches."""
    rows = [i % 4 for i in range(2500)]
    _run(rows, [(i * 5) % 7 - 1 for i in range(2500)], 6, 16, 128, 128)


def test_no_rows():
    plan = tq.exl3_adapter_plan(_i32([0, 0]), _i32([0]), 0, 1)
    y = torch.empty((0, 128), device="cuda")
    x = torch.empty((0, 128), dtype=torch.float16, device="cuda")
    assert tq.exl3_adapter_add(x, y, tq.adapters(*_pool(1, 8, 128, 128)), plan) is y


@pytest.mark.parametrize("T,R,n", [(40, 16, 384), (300, 128, 8192)])
def test_plan_is_refilled_in_a_graph(T, R, n):
    """One captured graph (plan and two linears' adapters) follows changed starts and adapters."""
    k, N = 256, 4
    assert _large(T, R, n) == (T > 40)
    x = torch.randn((T, k), generator=_gen(1), device="cuda").half()
    y = torch.randn((T, n), generator=_gen(2), device="cuda").half()
    out, out2 = torch.empty_like(y), torch.empty_like(y)
    pool, pool2 = _pool(N, R, k, n), _pool(N, 64, k, n, seed=3)
    ad, ad2 = tq.adapters(*pool), tq.adapters(*pool2)
    q, ids = _i32([0, 10, 20, T]), _i32([0, 1, 2])
    plan = tq.exl3_adapter_plan(q, ids, T, N)

    def step():
        tq.exl3_adapter_plan(q, ids, T, N, plan=plan)
        tq.exl3_adapter_add(x, y, ad, plan, out=out)
        tq.exl3_adapter_add(x, y, ad2, plan, out=out2)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for rows, which in (([10, 10, T - 20], [0, 1, 2]), ([1, T - 2, 1], [3, 3, -1]), ([T, 0, 0], [2, 2, 1])):
        q.copy_(_i32(_starts(rows)))
        ids.copy_(_i32(which))
        g.replay()
        torch.cuda.synchronize()
        _check(out, *_reference(x, y, pool, rows, which))
        _check(out2, *_reference(x, y, pool2, rows, which))


@pytest.mark.parametrize("T,R,n", [(24, 16, 1024), (300, 128, 8192)])
def test_one_plan_on_two_streams(T, R, n):
    k, N = 512, 3
    x = torch.randn((T, k), generator=_gen(1), device="cuda").half()
    y = torch.randn((T, n), generator=_gen(2), device="cuda").half()
    pools = [_pool(N, R, k, n, seed=s) for s in (0, 1)]
    ads = [tq.adapters(*p) for p in pools]
    plan = tq.exl3_adapter_plan(_i32([0, 7, T]), _i32([2, 0]), T, N)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ads]
    outs = [torch.empty_like(y) for _ in ads]
    torch.cuda.synchronize()
    for _ in range(20):
        for a, s, o in zip(ads, streams, outs):
            with torch.cuda.stream(s):
                tq.exl3_adapter_add(x, y, a, plan, out=o)
    torch.cuda.synchronize()
    for p, o in zip(pools, outs):
        _check(o, *_reference(x, y, p, [7, T - 7], [2, 0]))


def test_bindings_refuse_mismatches():
    x, y = torch.zeros((4, 128), dtype=torch.float16, device="cuda"), torch.zeros((4, 256), device="cuda")
    pool = tq.adapters(*_pool(2, 8, 128, 256))
    plan = tq.exl3_adapter_plan(_i32([0, 4]), _i32([0]), 4, 2)
    with pytest.raises(ValueError, match="rows"):
        tq.exl3_adapter_add(x[:3], y, pool, plan)
    with pytest.raises(ValueError, match="adapters"):
        tq.exl3_adapter_add(x, y, tq.adapters(*_pool(3, 8, 128, 256)), plan)
    with pytest.raises(TypeError, match="x must be"):
        tq.exl3_adapter_add(x.float(), y, pool, plan)
    with pytest.raises(TypeError, match="out must be"):
        tq.exl3_adapter_add(x, y, pool, plan, out=y.half())
    with pytest.raises(ValueError, match="plan was made"):
        tq.exl3_adapter_plan(_i32([0, 4]), _i32([0]), 5, 2, plan=plan)


@pytest.mark.parametrize("T,batch,R,n", [(100000, 1, 8, 128), (40, 2, 8, 128), (70000, 1, 128, 256), (300, 3000, 128, 8192)])
def test_a_plan_of_another_call_is_recorded(T, batch, R, n):
    """The C entry point gets a plan that was made for six rows and is as long as these need: behind
    its control block nothing of it may be read by the sizes of this call."""
    k, L = 128, tq.lib()
    x = torch.zeros((T, k), dtype=torch.float16, device="cuda")
    y, out = torch.zeros((T, n), device="cuda"), torch.full((T, n), 7.0, device="cuda")
    pool = tq.adapters(*_pool(2, R, k, n))
    plan = tq.exl3_adapter_plan(_i32([0, 6]), _i32([1]), 6, 2)
    ws = torch.zeros(tq.exl3_adapter_add_workspace_size(T, R), dtype=torch.uint8, device="cuda")
    assert plan.data.numel() <= tq.exl3_adapter_plan_size(T, batch, 2)    # (whole blocks of 256 bytes)
    assert L.exl3_adapter_add(x.data_ptr(), k, y.data_ptr(), n, out.data_ptr(), n, tq.EXL3_OUT_F32, pool._address,
                              plan.address, T, batch, ws.data_ptr(), ws.numel(), None) == 0
    torch.cuda.synchronize()
    assert (out == 7).all() and tq.exl3_check_device_error(ws) != 0


def test_a_plan_of_another_device_is_refused():
    """(With one GPU: a plan that says so.)"""
    q, ids = _i32([0, 4]), _i32([0])
    plan = tq.exl3_adapter_plan(q, ids, 4, 2)
    plan.device += 1
    with pytest.raises(ValueError, match="plan is on"):
        tq.exl3_adapter_plan(q, ids, 4, 2, plan=plan)


def _captured(T, R, n, stream, named, plan=None, seed=1):
    """A captured call's graph, inputs and output."""
    k, N = 256, 2
    x = torch.randn((T, k), generator=_gen(seed), device="cuda").half()
    y = torch.randn((T, n), generator=_gen(seed + 1), device="cuda").half()
    pool = _pool(N, R, k, n, seed=seed)
    plan = plan or tq.exl3_adapter_plan(_i32([0, 7, T]), _i32([1, 0]), T, N)
    ad, out = tq.adapters(*pool), torch.empty_like(y)
    kw = dict(stream=stream) if named else {}
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        tq.exl3_adapter_add(x, y, ad, plan, out=out, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        for _ in range(3):
            tq.exl3_adapter_add(x, y, ad, plan, out=out, **kw)
    return g, (x, y, ad, plan, pool), out


@pytest.mark.parametrize("named", [False, True])
@pytest.mark.parametrize("T,R,n", [(24, 16, 1024), (300, 128, 8192)])
def test_a_graph_keeps_nothing_in_the_streams_workspace(T, R, n, named):
    """Two graphs captured on one stream would race there when they run at once: what a graph
    leaves in the stream's workspace is an error word at most."""
    s = torch.cuda.Stream()
    assert _large(T, R, n) == (tq.exl3_adapter_scratch_size(T, R, n) > 0) == (T > 24)
    g, (x, y, _, _, pool), out = _captured(T, R, n, s, named)
    with torch.cuda.stream(s):
        ws = tq.workspace(1)
    used = ws.clone()
    ws[33024:] = 0x77                                      # (all but the counters)
    g.replay()
    torch.cuda.synchronize()
    assert (ws[33024:] == 0x77).all() and not ws[:33024].any()
    ws.copy_(used)
    _check(out, *_reference(x, y, pool, [7, T - 7], [1, 0]))


@pytest.mark.parametrize("named", [False, True])
@pytest.mark.parametrize("T,R,n", [(300, 128, 8192), (2500, 64, 2048)])
def test_two_graphs_of_one_stream_at_once(T, R, n, named):
    s = torch.cuda.Stream()
    made = [_captured(T, R, n, s, named, seed=seed) for seed in (1, 5)]
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, _, _), on in zip(made, streams):
            with torch.cuda.stream(on):
                g.replay()
    torch.cuda.synchronize()
    for _, (x, y, _, _, pool), out in made:
        _check(out, *_reference(x, y, pool, [7, T - 7], [1, 0]))


@pytest.mark.parametrize("named", [False, True])
@pytest.mark.parametrize("T,R,n", [(24, 16, 1024), (300, 128, 8192)])
def test_errors_of_a_graph_are_found_in_its_streams_workspace(T, R, n, named):
    """A plan that was never filled, found when the graph runs."""
    s = torch.cuda.Stream()
    g, _, out = _captured(T, R, n, s, named, plan=tq.AdapterPlan(T, 2, 2, "cuda"))
    with torch.cuda.stream(s):
        ws = tq.workspace(1)
        assert tq.exl3_check_device_error(ws) != 0         # (the call before the capture)
        assert tq.exl3_check_device_error(ws) == 0
        out.fill_(7.0)
        g.replay()
        assert tq.exl3_check_device_error(ws) != 0
    assert (out == 7).all()


@pytest.mark.parametrize("T,R,n", [(24, 16, 1024), (300, 128, 8192)])
def test_scratch_apart_from_the_error_word(T, R, n):
    k, need = 256, tq.exl3_adapter_scratch_size(T, R, n)
    x = torch.randn((T, k), generator=_gen(1), device="cuda").half()
    y = torch.randn((T, n), generator=_gen(2), device="cuda")
    pool = _pool(2, R, k, n)
    ad, plan = tq.adapters(*pool), tq.exl3_adapter_plan(_i32([0, 7, T]), _i32([1, 0]), T, 2)
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    buf = torch.full((need + 512,), 0x77, dtype=torch.uint8, device="cuda")
    out = tq.exl3_adapter_add_scratch(x, y, ad, plan, buf[:need] if need else None, out=torch.empty_like(y),
                                      workspace_buf=ws)
    _check(out, *_reference(x, y, pool, [7, T - 7], [1, 0]))
    assert (buf[need:] == 0x77).all() and not ws.any()
    assert torch.equal(out, tq.exl3_adapter_add(x, y, ad, plan, out=torch.empty_like(y)))
    if need:
        with pytest.raises(tq.Exl3Error, match="needed"):
            tq.exl3_adapter_add_scratch(x, y, ad, plan, buf[:need - 1], out=out, workspace_buf=ws)
        with pytest.raises(tq.Exl3Error, match="scratch is NULL"):
            tq.exl3_adapter_add_scratch(x, y, ad, plan, None, out=out, workspace_buf=ws)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("T,R,n", [(1, 16, 256), (8, 64, 256), (9, 16, 256), (40, 128, 384), (140, 24, 256), (140, 128, 16384)])
def test_infinities_in_x(T, R, n, fp32):
    """What the formula gives: +-infinity with one rank, and with ranks of one sign; NaN for infinity
    times zero; other rows as they were."""
    assert _large(T, R, n) == (n > 1000)
    k, N = 256, 3
    a, b, scale, _ = _pool(N, R, k, n)
    a[1], b[1] = a[1].abs() + 2.0 ** -10, b[1].abs() + 2.0 ** -10
    a[0] = torch.where(a[0].abs() < 2.0 ** -10, torch.full_like(a[0], 2.0 ** -10), a[0])
    a[2] = 0.0                                             # (infinity times zero)
    b[0] = torch.where(b[0].abs() < 2.0 ** -10, torch.full_like(b[0], 2.0 ** -10), b[0])
    ranks = [1, R, R]
    pool = (a, b, scale, _i32(ranks))
    for i, r in enumerate(ranks[:2]):
        a[i, r:], b[i, :, r:] = 0, 0
    x = torch.randn((T, k), generator=_gen(1), device="cuda").half()
    y = torch.randn((T, n), generator=_gen(2), device="cuda").to(torch.float32 if fp32 else torch.float16)
    third = T // 3
    rows, ids = ([T], [0]) if T == 1 else ([third, third, T - 2 * third], [0, 1, 2])
    plan, ad = tq.exl3_adapter_plan(_i32(_starts(rows)), _i32(ids), T, N), tq.adapters(*pool)
    clean = tq.exl3_adapter_add(x, y, ad, plan, out=torch.empty_like(y))
    bad = [0] if T == 1 else [0, third, T - 1]
    x[bad[0], 7] = math.inf
    if T > 1:
        x[bad[1], 9] = -math.inf
        x[bad[2], 11] = math.inf
    got = tq.exl3_adapter_add(x, y, ad, plan, out=torch.empty_like(y))
    for t, i in zip(bad, ids):
        A, B = a[i, :ranks[i]].double(), b[i, :, :ranks[i]].double()
        h = (x[t].double() * A).sum(-1)
        want = (y[t].double() + float(scale[i]) * (h * B).sum(-1)).to(y.dtype)
        assert torch.equal(got[t].isnan(), want.isnan()) and torch.equal(got[t].nan_to_num(0.5), want.nan_to_num(0.5))
        assert want.isnan().all() if i == 2 else want.isinf().all()
    rest = [t for t in range(T) if t not in bad]
    assert torch.equal(got[rest], clean[rest])


@pytest.mark.parametrize("T,R,n", [(5, 16, 256), (12, 16, 256), (140, 128, 16384)])
def test_finite_ranks_beside_an_infinite_one(T, R, n):
    """h = (infinity, 1e6 of either sign): the finite one is above fp16's range and adds nothing."""
    assert _large(T, R, n) == (n > 1000)
    k = 128
    a = torch.zeros((1, R, k), dtype=torch.float16, device="cuda")
    b = torch.ones((1, n, R), dtype=torch.float16, device="cuda")
    a[0, :, 0] = 60000.0                                   # every rank 60000 * 60000 * 2 in each row,
    a[0, 1::2, 0] = -60000.0
    x = torch.zeros((T, k), dtype=torch.float16, device="cuda")
    x[:, 0] = 60000.0
    y = torch.zeros((T, n), device="cuda")
    scale = torch.ones(1, device="cuda")
    plan, ad = tq.exl3_adapter_plan(_i32([0, T]), _i32([0]), T, 1), tq.adapters(a, b, scale)
    got = tq.exl3_adapter_add(x, y, ad, plan, out=torch.empty_like(y))
    assert (got == 0).all()                                # which cancel
    a[0, 2, 1] = math.inf                                  # and one of them infinite where x has a 1
    a[0, :, 1] = torch.where(a[0, :, 1].isinf(), a[0, :, 1], torch.zeros_like(a[0, :, 1]))
    x[T // 2, 1] = 1.0
    x[:T // 2, 1] = 0.25
    x[T // 2 + 1:, 1] = -2.0
    got = tq.exl3_adapter_add(x, y, tq.adapters(a, b, scale), plan, out=torch.empty_like(y))
    assert (got[:T // 2 + 1] == math.inf).all() and (got[T // 2 + 1:] == -math.inf).all()
