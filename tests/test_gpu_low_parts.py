"""The low parts of values that are held as two fp16 numbers: packed router weights, and h of the
adapters' second product.

The tolerances of the other tests grow with the sums and hide a low part that is missing or comes
from the wrong place.  Here every output is one such value: an odd integer of 22 bits, which two
parts of 11 hold exactly and one does not, alone in its sum.  So outputs are equal, bit for bit."""
import pytest
import torch

import trellis_quantized_gb300 as tq


def _odd(shape, seed):
    """Odd integers of 22 bits, of either sign, as float32, with their factors 2048 p + q (q odd)."""
    g = torch.Generator()
    g.manual_seed(seed)
    p = torch.randint(1024, 2048, shape, generator=g)
    q = 2 * torch.randint(0, 1024, shape, generator=g) + 1
    sign = 2 * torch.randint(0, 2, shape, generator=g) - 1
    return (sign * (2048 * p + q)).float(), (sign * p).half(), (sign * q).half()


def _parts(v, low=True):
    """v in two fp16 parts after a power of two, put together again; `low` false: without the second."""
    z = v.double() * 2.0 ** -7
    hi = z.half().double()
    lo = ((z - hi) * 2048).half().double() / 2048 if low else 0.0
    return (hi + lo) * 2.0 ** 7


def test_the_values_need_their_low_parts():
    """Two parts hold each of them, one holds none."""
    v, p, q = _odd((20000,), 0)
    assert torch.equal(2048 * p.double() + q.double(), v.double())
    assert torch.equal(_parts(v), v.double()) and (_parts(v, low=False) != v.double()).all()


# ------------------------------------------------------------------- router

@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 5, 8, 9, 64, 200, 1333])
@pytest.mark.parametrize("k,E", [(128, 8), (5120, 60), (2048, 256), (1048, 300), (8192, 130), (520, 1)])
def test_packed_router_weights(T, k, E):
    """Row t of x has a single 1, in another block of 64 than the row before it: its logits are a column of w."""
    w = _odd((E, k), 1)[0].cuda()
    at = torch.arange(T, device="cuda") * 67 % k
    x = torch.zeros((T, k), dtype=torch.float16, device="cuda")
    x[torch.arange(T, device="cuda"), at] = 1
    assert torch.equal(tq.exl3_router_logits(x, tq.router(w)), w.t()[at])


@pytest.mark.gpu
def test_router_columns_one_after_another():
    """Every column of k, at more rows than one tile has."""
    k, E = 2560, 132
    w = _odd((E, k), 2)[0].cuda()
    x = torch.eye(k, dtype=torch.float16, device="cuda")
    assert torch.equal(tq.exl3_router_logits(x, tq.router(w)), w.t())


# ----------------------------------------------------------------- adapters

def _adapt(rows, R, k, n, ranks=None):
    """h[t, r] = 2048 p + q from two places of k, which change with t; column c of B takes rank c % R alone."""
    N, T = 2, sum(rows)
    a = torch.zeros((N, R, k), dtype=torch.float16, device="cuda")
    v, p, q = _odd((N, k // 2, R), 3)                      # (place j of either half of k has values of its own)
    a[:, :, :k // 2] = p.cuda().transpose(1, 2)
    a[:, :, k // 2:] = q.cuda().transpose(1, 2)
    j = torch.arange(T, device="cuda") * 67 % (k // 2)
    x = torch.zeros((T, k), dtype=torch.float16, device="cuda")
    t = torch.arange(T, device="cuda")
    x[t, j], x[t, j + k // 2] = 2048.0, 1.0
    b = torch.zeros((N, n, R), dtype=torch.float16, device="cuda")
    c = torch.arange(n, device="cuda")
    b[:, c, c % R] = 1
    owner = torch.tensor([i % N for i in range(len(rows)) for _ in range(rows[i])], device="cuda")
    h = v.cuda()[owner, j]                                 # [T, R]
    rank = None
    if ranks is not None:
        rank = torch.tensor(ranks, dtype=torch.int32, device="cuda")
        h = torch.where(torch.arange(R, device="cuda")[None] < rank[owner.long()][:, None], h, 0.0)
    starts = [0]
    for r in rows:
        starts.append(starts[-1] + r)
    plan = tq.exl3_adapter_plan(torch.tensor(starts, dtype=torch.int32, device="cuda"),
                                torch.tensor([i % N for i in range(len(rows))], dtype=torch.int32, device="cuda"), T, N)
    pool = tq.adapters(a, b, torch.ones(N, device="cuda"), rank=rank)
    y = torch.zeros((T, n), device="cuda")
    out = tq.exl3_adapter_add(x, y, pool, plan, out=torch.empty_like(y))
    assert torch.equal(out, h[:, c % R])
    return T, R, n


@pytest.mark.gpu
@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 72, 104, 128])
@pytest.mark.parametrize("rows", [[1], [5], [8], [9], [16], [3, 17, 1, 12]])
@pytest.mark.parametrize("k,n", [(128, 384), (8192, 640)])
def test_h_on_tiles_of_16_rows(rows, R, k, n):
    T, R, n = _adapt(rows, R, k, n)
    assert tq.exl3_adapter_scratch_size(T, R, n) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("R,n", [(8, 49792), (16, 28032), (24, 17920), (40, 9216), (64, 4480), (72, 3712), (104, 2048),
                                 (128, 1408)])
@pytest.mark.parametrize("rows", [[600], [200, 1, 333, 2, 64]])
@pytest.mark.parametrize("k", [256, 4096])
def test_h_on_tiles_of_128_rows(rows, R, n, k):
    T, R, n = _adapt(rows, R, k, n)
    assert tq.exl3_adapter_scratch_size(T, R, n) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("rows,n", [([9], 384), ([600, 40], 2048)])
def test_h_up_to_an_adapters_rank(rows, n):
    _adapt(rows, 128, 512, n, ranks=[77, 100])
