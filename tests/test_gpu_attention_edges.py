"""exl3_paged_attention where it can go wrong: units of one block, extreme
scores, one key that outweighs a long history, batches whose sequences differ
most.  Helpers and bounds are those of tests/test_gpu_attention.py and
tests/attention_ref.py, unless a test derives a closer bound of its own."""
import pytest
import torch

import trellis_quantized_gb300 as tq
from attention_ref import U16, U32
from test_gpu_attention import _compare, _run, _setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,rows", [(16, 2, 3), (8, 8, 20), (128, 1, 1)])
@pytest.mark.parametrize("B", [1, 30, 160])
def test_units_of_one_block(Hq, Hkv, rows, B):
    """256-wide heads on the tensor cores: every unit has one block of 64 keys, or
    (every fifth sequence) two, so that the two score warps take turns."""
    old = [(i * 13) % (60 - rows) + (64 if i % 5 == 4 else 0) for i in range(B)]
    _run([rows] * B, old, Hq, Hkv, 256)


@pytest.mark.parametrize("rows", [40, 17])
def test_short_units_among_long_ones(rows):
    """256-wide heads: units of one block between units that are cut."""
    old = [0, 9000, 1, 5, 20, 3000, 0, 0, 0, 15, 64, 2, 7000]
    _run([rows] * len(old), old, 8, 4, 256, page=32)


def _signs(shape, size, gen):
    return (torch.randint(0, 2, shape, generator=gen, device="cuda") * 2 - 1).half() * size


def _sign_scores(new, old, Hq, Hkv, D, size, page=16):
    """Attention with q and k of +-size in every element.  A score is then an
    integer times size^2 with at most 24 significant bits, so every product and
    sum of it is exact in fp32; scores that differ do so by 2 size^2 at least,
    which leaves weights of zero: y is the mean of v over a row's largest keys.
    Returns y, lse, the exact means, the keys of each mean and the exact lse."""
    q, k, v, table, dense, q_start, kv_len = _setup([new], [old], Hq, Hkv, D, page, "tokens", seed=3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(new + old + D)
    q.copy_(_signs(q.shape, size, gen))
    kd, vd = dense[0]
    kd.copy_(_signs(kd.shape, size, gen))
    p = torch.arange(new + old, device="cuda")
    k[table[0].long()[p // page], p % page] = kd
    lse = torch.empty((new, Hq), dtype=torch.float32, device="cuda")
    ws = torch.zeros(tq.exl3_paged_attention_workspace_size(new, Hq, Hkv, D, 1), dtype=torch.uint8, device="cuda")
    y = tq.exl3_paged_attention(q, tq.paged_batch(q_start, kv_len, table), tq.kv_cache(k, v), lse=lse, workspace_buf=ws)
    assert tq.exl3_check_device_error(ws) == 0
    G = Hq // Hkv
    s = torch.einsum("tgd,jgd->tgj", q.double(), kd.double().repeat_interleave(G, 1))
    s = torch.where(p[None, None, :] <= old + torch.arange(new, device="cuda")[:, None, None], s, -torch.inf)
    top = s.amax(-1, keepdim=True)
    largest = (s == top).double()
    keys = largest.sum(-1)
    mean = torch.einsum("tgj,jgd->tgd", largest, vd.double().repeat_interleave(G, 1)) / keys[..., None]
    size_of_terms = torch.einsum("tgj,jgd->tgd", largest, vd.double().abs().repeat_interleave(G, 1)) / keys[..., None]
    return y, lse, mean, size_of_terms, keys, top[..., 0] * D ** -0.5 + torch.log(keys)


def _compare_means(y, lse, mean, terms, want_lse, rows):
    """One rounding of y to fp16; sums of at most some tens of terms, the
    division and the exponential of the weights within 2^-20 of the terms; an
    lse within eight roundings of its size (scale, its product with the
    maximum, the natural logarithm's factor, the sum)."""
    assert torch.isfinite(y).all() and torch.isfinite(lse).all()
    bound = U16 * mean.abs() + 2.0 ** -25 + 2.0 ** -20 * terms
    assert ((y.double() - mean).abs() <= bound)[rows].all()
    assert ((lse.double() - want_lse).abs() <= 2.0 ** -21 * want_lse.abs())[rows].all()


@pytest.mark.parametrize("size", [8000.0, 32768.0])
@pytest.mark.parametrize("Hq,Hkv,D", [(40, 8, 128), (16, 2, 256), (24, 8, 64)])
@pytest.mark.parametrize("new,old", [(1, 700), (100, 700), (300, 0)])
def test_scores_of_any_size(size, Hq, Hkv, D, new, old):
    """Scores up to 2^37: rows with one largest key have its v, all rows are finite."""
    y, lse, mean, terms, keys, want_lse = _sign_scores(new, old, Hq, Hkv, D, size)
    _compare_means(y, lse, mean, terms, want_lse, keys == 1)


@pytest.mark.parametrize("size", [8000.0, 32768.0])
@pytest.mark.parametrize("Hq,Hkv,D", [(40, 8, 128), (16, 2, 256), (24, 8, 64)])
@pytest.mark.parametrize("new,old", [(1, 700), (1, 5000), (100, 700)])
def test_ties_at_scores_of_any_size(size, Hq, Hkv, D, new, old):
    """Largest keys in several parts of a cut sequence, in different numbers: each counts once."""
    y, lse, mean, terms, keys, want_lse = _sign_scores(new, old, Hq, Hkv, D, size)
    assert (keys > 1).any()
    _compare_means(y, lse, mean, terms, want_lse, keys >= 1)


@pytest.mark.parametrize("D,G,new,B,smallest", [
    (128, 4, 1, 700, 2.0 ** -40), (64, 7, 2, 900, 2.0 ** -40), (256, 8, 1, 300, 2.0 ** -40),
    (128, 4, 8, 300, 2.0 ** -32), (64, 40, 7, 150, 2.0 ** -32), (256, 8, 5, 300, 2.0 ** -32)])
def test_a_key_that_outweighs_a_long_history(D, G, new, B, smallest):
    """A first key at weight 1 whose value is zero, 131,072 others at 2^-24 to
    2^-25.5 of it: all of y is their share.  B sequences read the same pages, so
    that most units stay whole.  Scores are single products, exact in fp32; the
    bound has the terms of attention_ref without the dot product's, and takes
    the smallest weight that is held (2^-25 fp16 steps below the largest,
    which lies at 2^15 in the step kernel and at 2^7 or more in the other)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(D + G + new)
    page, L = 256, 131072 + 256
    rand = lambda *shape: torch.rand(shape, generator=gen, device="cuda")
    k = torch.zeros((L, 1, D), dtype=torch.float16, device="cuda")
    k[:, 0, 0] = -(16.64 + 1.03 * rand(L)).half()
    k[0, 0, 0] = 0
    v = (0.5 + rand(L, 1, D)).half()
    v[0] = 0
    q = torch.zeros((B * new, G, D), dtype=torch.float16, device="cuda")
    q[:, :, 0] = (0.97 + 0.03 * rand(B * new, G)).half()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table = torch.arange(L // page, dtype=torch.int32, device="cuda").repeat(B, 1)
    batch = tq.paged_batch(i32(range(0, B * new + 1, new)), i32([L] * B), table)
    cache = tq.kv_cache(k.view(-1, page, 1, D), v.view(-1, page, 1, D))
    lse = torch.empty((B * new, G), dtype=torch.float32, device="cuda")
    y = tq.exl3_paged_attention(q, batch, cache, scale=1.0, out_dtype=tq.EXL3_OUT_F32, lse=lse)
    rows = range(0, B * new, max(1, B * new // 60))
    for t in rows:
        n = L - new + t % new + 1
        s = q[t, :, 0].double()[:, None] * k[:n, 0, 0].double()[None]
        p = torch.exp(s)
        l = p.sum(1, keepdim=True)
        want = p @ v[:n, 0].double() / l
        ds = 4 * U32 * 17.7 + 2.0 ** -20
        bound = (2 * ds + U16 + (L / 16 + 64) * U32) * want + L * smallest * 1.5 / l + U32 * want
        err = (y[t].double() - want).abs()
        assert (err <= bound).all(), f"row {t}: worst error / bound {(err / bound).max().item():.3f}"
        want_lse = torch.log(l[:, 0])
        assert ((lse[t].double() - want_lse).abs() <= 2 * ds + (L / 16 + 64) * U32 + 2.0 ** -22 * want_lse.abs()).all()


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 8, 128), (16, 2, 256), (24, 8, 64)])
@pytest.mark.parametrize("new,old", [(1, 20), (1, 900), (2, 300), (60, 200)])
def test_nan_stays_where_it_is_seen(Hq, Hkv, D, new, old):
    """A NaN in a query makes its row's y and lse NaN and no other's; so do NaN
    keys for the rows that see them, whole groups of 16 keys among them."""
    q, k, v, table, dense, q_start, kv_len = _setup([new], [old], Hq, Hkv, D, 16, "tokens", seed=9)
    args = (tq.paged_batch(q_start, kv_len, table), tq.kv_cache(k, v))
    lse = torch.empty((new, Hq), dtype=torch.float32, device="cuda")
    qn = q.clone()
    qn[0, 1, 5] = torch.nan
    y = tq.exl3_paged_attention(qn, *args, lse=lse)
    assert torch.isnan(y[0, 1]).all() and torch.isnan(lse[0, 1])
    y0 = tq.exl3_paged_attention(q, *args)
    y[0, 1] = y0[0, 1]
    _compare(y, None, q, dense, [new], [old], True, 0, D ** -0.5)
    assert torch.isnan(lse).sum() == 1
    for first, count in ((old, 1), (0, 16)):           # the first new key; a whole page of keys
        p = torch.arange(first, first + count, device="cuda")
        kn = k.clone()
        kn[table[0].long()[p // 16], p % 16] = torch.nan
        y = tq.exl3_paged_attention(q, args[0], tq.kv_cache(kn, v), lse=lse)
        assert torch.isnan(y).all() and torch.isnan(lse).all()
        if new > 1:                                    # a key that only the last row sees
            kn = k.clone()
            kn[table[0, (old + new - 1) // 16], (old + new - 1) % 16] = torch.nan
            y = tq.exl3_paged_attention(q, args[0], tq.kv_cache(kn, v), lse=lse)
            assert torch.isnan(y[-1]).all() and torch.isnan(lse[-1]).all()
            assert not torch.isnan(y[:-1]).any() and not torch.isnan(lse[:-1]).any()


@pytest.mark.parametrize("B,at", [(30, 0), (30, 29), (64, 63), (150, 70)])
@pytest.mark.parametrize("Hq,Hkv,D,chunk,behind", [(40, 8, 128, 141, 900), (8, 8, 128, 400, 300), (16, 2, 256, 60, 2000),
                                                   (24, 8, 64, 333, 0)])
def test_one_chunk_among_many_steps(B, at, Hq, Hkv, D, chunk, behind):
    """One-token sequences before, around and behind a chunk of many units, with few
    enough rows in all for the step kernel (where they are too many, on the tensor cores):
    the chunk's units are counted, found and shared out."""
    new, old = [1] * B, [(i * 29) % 150 for i in range(B)]
    new[at], old[at] = chunk, behind
    _run(new, old, Hq, Hkv, D)
