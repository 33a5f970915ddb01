"""GPU parity of exl3_paged_attention against the plain 64-bit form.  The cache
holds NaN and infinities wherever no row of the call looks, and table entries
that no row needs are -1.  Bounds are derived in tests/attention_ref.py."""
import math

import pytest
import torch

import trellis_quantized_gb300 as tq
from attention_ref import U16, attention, paged

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(new):
    s = [0]
    for n in new:
        s.append(s[-1] + n)
    return s


def _setup(new, old, Hq, Hkv, D, page, order, window=0, seed=0, q_scale=2.0, interleaved=False, pad=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + sum(new) * 31 + sum(old) + D)
    lens = [n + o for n, o in zip(new, old)]
    first = [max(0, o - window + 1) if window else 0 for o in old]
    k, v, table, dense = paged(lens, page, Hkv, D, order, gen, first, interleaved=interleaved)
    T = sum(new) + pad
    q = (q_scale * torch.randn((T, Hq, D), generator=gen, device="cuda")).half()
    return q, k, v, table, dense, _i32(_starts(new)), _i32(lens)


def _compare(y, lse, q, dense, new, old, causal, window, scale):
    t = 0
    for b, (n, o) in enumerate(zip(new, old)):
        if n:
            kd, vd = dense[b]
            wy, wl, by, bl = attention(q[t:t + n], kd, vd, o, causal, window, scale)
            gy = y[t:t + n].double()
            bound = by + (U16 * wy.abs() + 2.0 ** -25 if y.dtype == torch.float16 else 2.0 ** -24 * wy.abs())
            err = (gy - wy).abs()
            assert torch.isfinite(gy).all(), f"sequence {b}: non-finite output"
            assert (err <= bound).all(), f"sequence {b}: worst error / bound {(err / bound.clamp_min(1e-300)).max():.3f}"
            if lse is not None:
                gl = lse[t:t + n].double()
                dead = torch.isinf(wl)
                assert (gl[dead] == -math.inf).all()
                assert ((gl - wl).abs()[~dead] <= bl[~dead]).all(), f"sequence {b}: lse"
        t += n


def _run(new, old, Hq, Hkv, D, page=16, order="tokens", causal=True, window=0, out=tq.EXL3_OUT_F16, scale=None,
         seed=0, interleaved=False, pad=0):
    q, k, v, table, dense, q_start, kv_len = _setup(new, old, Hq, Hkv, D, page, order, window, seed,
                                                    interleaved=interleaved, pad=pad)
    T = q.shape[0]
    lse = torch.empty((T, Hq), dtype=torch.float32, device="cuda")
    ws = torch.zeros(tq.exl3_paged_attention_workspace_size(T, Hq, Hkv, D, len(new)), dtype=torch.uint8, device="cuda")
    y = tq.exl3_paged_attention(q, tq.paged_batch(q_start, kv_len, table), tq.kv_cache(k, v), scale=scale,
                                causal=causal, window=window, out_dtype=out, lse=lse, workspace_buf=ws)
    assert tq.exl3_check_device_error(ws) == 0
    assert not ws[:256 + 4 * 8192].any(), "counters are zero again"
    _compare(y, lse, q, dense, new, old, causal, window, D ** -0.5 if scale is None else scale)
    if pad:
        assert not y[T - pad:].any() and (lse[T - pad:] == -math.inf).all()
    return y


HEADS = [(40, 8, 128), (16, 2, 256), (24, 8, 64), (8, 8, 128), (7, 1, 128), (32, 1, 64), (100, 1, 128)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("old", [0, 1, 15, 16, 63, 64, 127, 500, 3001])
def test_one_token(Hq, Hkv, D, old):
    _run([1], [old], Hq, Hkv, D)


@pytest.mark.parametrize("page", [16, 48, 64, 80, 128, 256])
@pytest.mark.parametrize("order", ["tokens", "heads"])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS[:3])
def test_page_sizes_and_orders(page, order, Hq, Hkv, D):
    _run([1, 1, 3], [200, 77, 1000], Hq, Hkv, D, page=page, order=order)


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_ragged_steps(Hq, Hkv, D):
    old = [0, 5, 4096, 33, 900, 17, 1, 2047, 64, 128, 3, 700]
    _run([1] * len(old), old, Hq, Hkv, D)


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("new,old", [([2], [0]), ([5, 3, 16], [100, 0, 777]), ([17, 1, 40], [0, 300, 129]),
                                     ([128], [0]), ([129], [63]), ([300, 1, 0, 77], [0, 500, 40, 1000]),
                                     ([257, 255], [511, 0])])
def test_chunks(Hq, Hkv, D, new, old):
    _run(new, old, Hq, Hkv, D)


@pytest.mark.parametrize("Hq,Hkv,D", HEADS[:3])
@pytest.mark.parametrize("window", [1, 2, 17, 64, 129, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("new,old", [([1, 1], [600, 3]), ([200, 30], [450, 0])])
def test_windows(Hq, Hkv, D, window, new, old):
    _run(new, old, Hq, Hkv, D, window=window, page=32)


@pytest.mark.parametrize("Hq,Hkv,D", HEADS[:3])
@pytest.mark.parametrize("new,old", [([1, 1], [600, 3]), ([200, 30], [450, 0])])
def test_not_causal(Hq, Hkv, D, new, old):
    _run(new, old, Hq, Hkv, D, causal=False)


@pytest.mark.parametrize("new,old", [([3, 1], [200, 40]), ([150], [130])])
def test_fp32_output_scale_and_one_allocation(new, old):
    _run(new, old, 40, 8, 128, out=tq.EXL3_OUT_F32, scale=0.03, interleaved=True)
    _run(new, old, 16, 2, 256, out=tq.EXL3_OUT_F32, scale=0.2, page=64, order="heads", interleaved=True)


@pytest.mark.parametrize("new", [[1, 0, 1], [40, 0, 3]])
def test_empty_sequences_and_padding_rows(new):
    _run(new, [10, 0, 300], 40, 8, 128, pad=5)


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 40, 8), (256, 16, 2)])
@pytest.mark.parametrize("n", [1, 60])
def test_long(D, Hq, Hkv, n):
    _run([n, n], [40000, 7], Hq, Hkv, D, page=64)


@pytest.mark.parametrize("n", [1, 50])
def test_large_scores(n):
    """Scores of hundreds: the running maximum rescales, nothing overflows."""
    q, k, v, table, dense, q_start, kv_len = _setup([n], [700], 8, 2, 128, 16, "tokens", q_scale=40.0)
    lse = torch.empty((n, 8), dtype=torch.float32, device="cuda")
    y = tq.exl3_paged_attention(q, tq.paged_batch(q_start, kv_len, table), tq.kv_cache(k, v), scale=1.0, lse=lse)
    _compare(y, lse, q, dense, [n], [700], True, 0, 1.0)


@pytest.mark.parametrize("n", [1, 100])
def test_rising_scores(n):
    """Keys that grow along the sequence: every block raises the maximum."""
    q, k, v, table, dense, q_start, kv_len = _setup([n], [1500], 8, 2, 64, 16, "tokens")
    L = n + 1500
    ramp = torch.linspace(0.0, 30.0, L, device="cuda")
    kd = dense[0][0]
    kd.copy_((ramp[:, None, None] + 0 * kd.float()).half())
    p = torch.arange(L, device="cuda")
    k[table[0].long()[p // 16], p % 16] = kd
    q.copy_(q.abs())
    lse = torch.empty((n, 8), dtype=torch.float32, device="cuda")
    y = tq.exl3_paged_attention(q, tq.paged_batch(q_start, kv_len, table), tq.kv_cache(k, v), lse=lse)
    _compare(y, lse, q, dense, [n], [1500], True, 0, 64 ** -0.5)


@pytest.mark.parametrize("new,old", [([1, 2], [300, 20]), ([90], [33])])
def test_strided_queries_other_stream_and_repeat(new, old):
    q, k, v, table, dense, q_start, kv_len = _setup(new, old, 40, 8, 128, 16, "tokens")
    T = q.shape[0]
    wide = torch.full((T, 40 * 128 + 2048), math.nan, dtype=torch.float16, device="cuda")
    wide[:, 1024:1024 + 5120] = q.reshape(T, -1)
    qs = wide[:, 1024:1024 + 5120].view(T, 40, 128)
    args = (tq.paged_batch(q_start, kv_len, table), tq.kv_cache(k, v))
    y0 = tq.exl3_paged_attention(q, *args)
    y1 = tq.exl3_paged_attention(qs, *args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y2 = tq.exl3_paged_attention(qs, *args)
    s.synchronize()
    assert torch.equal(y0, y1) and torch.equal(y0, y2)
    _compare(y0, None, q, dense, new, old, True, 0, 128 ** -0.5)


@pytest.mark.parametrize("out", [tq.EXL3_OUT_F16, tq.EXL3_OUT_F32])
@pytest.mark.parametrize("new,old", [([1, 2], [300, 20]), ([90, 300], [33, 0])])
def test_buffers_on_16_byte_boundaries(new, old, out):
    """q, y and the cache start 16 bytes past a 32-byte boundary."""
    q, k, v, table, dense, q_start, kv_len = _setup(new, old, 16, 2, 128, 16, "tokens")
    dt = torch.float32 if out == tq.EXL3_OUT_F32 else torch.float16

    def shifted(t, dtype):
        per16 = 16 // torch.empty(0, dtype=dtype).element_size()
        buf = torch.zeros(t.numel() + 2 * per16, dtype=dtype, device="cuda")
        off = per16 if buf.data_ptr() % 32 == 0 else 2 * per16
        return buf[off:off + t.numel()].view(t.shape)

    qs, ks, vs, ys = shifted(q, torch.float16), shifted(k, torch.float16), shifted(v, torch.float16), shifted(q, dt)
    qs.copy_(q), ks.copy_(k), vs.copy_(v)
    assert all(t.data_ptr() % 32 == 16 for t in (qs, ks, vs, ys))
    tq.exl3_paged_attention(qs, tq.paged_batch(q_start, kv_len, table), tq.kv_cache(ks, vs), out_dtype=out, y=ys)
    _compare(ys, None, q, dense, new, old, True, 0, 128 ** -0.5)


@pytest.mark.parametrize("n", [1, 40])
def test_graph_with_growing_lengths(n):
    """One captured call serves lengths that change between replays."""
    new, old = [n, n], [700, 300]
    q, k, v, table, dense, q_start, kv_len = _setup(new, old, 16, 2, 256, 32, "heads")
    batch, cache = tq.paged_batch(q_start, kv_len, table), tq.kv_cache(k, v)
    y = torch.empty_like(q)
    ws = torch.zeros(tq.exl3_paged_attention_workspace_size(2 * n, 16, 2, 256, 2), dtype=torch.uint8, device="cuda")
    tq.exl3_paged_attention(q, batch, cache, y=y, workspace_buf=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tq.exl3_paged_attention(q, batch, cache, y=y, workspace_buf=ws)
    for cut in ([0, 0], [500, 1], [699, 299], [3, 290]):
        lens = [n + o - c for o, c in zip(old, cut)]
        kv_len.copy_(_i32(lens))
        y.fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        _compare(y, None, q, [(kd[:L], vd[:L]) for (kd, vd), L in zip(dense, lens)], new,
                 [o - c for o, c in zip(old, cut)], True, 0, 256 ** -0.5)
    assert tq.exl3_check_device_error(ws) == 0


@pytest.mark.parametrize("n", [1, 40])
def test_bad_pages_and_lengths_are_reported(n):
    """A page outside the cache reads as zeros, lengths past the table are
    clamped, rows at negative indexes see nothing; each sets the error word."""
    q, k, v, table, dense, q_start, kv_len = _setup([n], [100], 8, 2, 128, 16, "tokens")
    ws = torch.zeros(tq.exl3_paged_attention_workspace_size(n, 8, 2, 128, 1), dtype=torch.uint8, device="cuda")
    cache = tq.kv_cache(k, v)
    for bad in (-1, k.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = bad
        y = tq.exl3_paged_attention(q, tq.paged_batch(q_start, kv_len, t), cache, workspace_buf=ws)
        assert tq.exl3_check_device_error(ws) != 0
        assert tq.exl3_check_device_error(ws) == 0
        kd, vd = dense[0][0].clone(), dense[0][1].clone()
        kd[32:48], vd[32:48] = 0, 0
        _compare(y, None, q, [(kd, vd)], [n], [100], True, 0, 128 ** -0.5)
    cap = table.shape[1] * 16
    full = torch.arange(table.shape[1], dtype=torch.int32, device="cuda")[None] % k.shape[0]
    clean_k, clean_v = torch.zeros_like(k), torch.zeros_like(v)
    y = tq.exl3_paged_attention(q, tq.paged_batch(q_start, _i32([cap + 1]), full.contiguous()),
                                tq.kv_cache(clean_k, clean_v), workspace_buf=ws)
    assert tq.exl3_check_device_error(ws) != 0 and not y.any()
    if n > 1:
        lse = torch.empty((n, 8), dtype=torch.float32, device="cuda")
        y = tq.exl3_paged_attention(q, tq.paged_batch(q_start, _i32([n - 3]), table), cache, workspace_buf=ws, lse=lse)
        assert tq.exl3_check_device_error(ws) != 0
        assert not y[:3].any() and (lse[:3] == -math.inf).all()
        _compare(y[3:], lse[3:], q[3:], [(dense[0][0][:n - 3], dense[0][1][:n - 3])], [n - 3], [0], True, 0, 128 ** -0.5)


def test_cache_past_two_gigabytes():
    """Pages whose offsets pass 2^31 elements and 2^32 bytes."""
    page, Hkv, D = 256, 8, 256
    pages = (2 ** 31 + 2 ** 26) // (page * Hkv * D) + 1
    k = torch.empty((pages, page, Hkv, D), dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    for n, L in ((1, 700), (50, 600)):
        table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
        kd = torch.randn((768, Hkv, D), generator=gen, device="cuda").half()
        vd = torch.randn((768, Hkv, D), generator=gen, device="cuda").half()
        for i in range(3):
            k[table[0, i].item()], v[table[0, i].item()] = kd[i * page:(i + 1) * page], vd[i * page:(i + 1) * page]
        q = torch.randn((n, 16, D), generator=gen, device="cuda").half()
        y = tq.exl3_paged_attention(q, tq.paged_batch(_i32([0, n]), _i32([L]), table), tq.kv_cache(k, v))
        _compare(y, None, q, [(kd[:L], vd[:L])], [n], [L - n], True, 0, D ** -0.5)


@pytest.mark.parametrize("B", [32, 33, 530])
@pytest.mark.parametrize("Hq,Hkv,D", [(10, 2, 128), (8, 1, 256)])
@pytest.mark.parametrize("chunks", [False, True])
def test_numbers_of_sequences(B, Hq, Hkv, D, chunks):
    """The work is found with and without block barriers; some sequences have no row, some no history."""
    old = [(i * 37) % 211 for i in range(B)]
    new = [(i * 5 + 3) % 41 for i in range(B)] if chunks else [1 - (i % 7 == 3) for i in range(B)]
    _run(new, old, Hq, Hkv, D, pad=3)


@pytest.mark.parametrize("B", [5, 34])
@pytest.mark.parametrize("rows", [1, 3, 9, 40, 41])
def test_joins_of_short_tiles(B, rows):
    """Long histories behind few rows: the units are cut, and their rows are spread over the join's blocks."""
    old = [4000 + 900 * (i % 3) for i in range(B)]
    _run([rows] * B, old, 16, 2, 256, page=64)
    _run([rows] * B, old, 20, 4, 128, page=64)
