"""Plain 64-bit forms of the attention operators (torch.float64 on the tensors'
device), the error bounds that their fp16/fp32 kernels have to keep, and
builders of paged caches whose unused places hold NaN and infinities.

Bounds.  u16 = 2^-11 and u32 = 2^-24 are half a step of fp16 and fp32.

* Head transform: about 8 + log2(D / 8) additions of squares, an rsqrt, the
  weights, the angle (2^-25 turns, i.e. 4 u32 of a unit vector) and a rotation:
  at most 32 u32 of the pair's size, then one rounding of the output (u16
  relative, 2^-25 absolute below fp16's normal range).
* Attention: a score is a dot product of D exact products accumulated in fp32
  (D u32 sum|q k|) scaled and subtracted from the maximum (4 u32 |s|), so a
  weight is off by ds = scale D u32 max sum|q k| + 4 u32 max|s| + 2^-20
  (exponential) + u16 (fp16 weights); weights below 2^-14 of the largest are
  subnormal fp16 values, off by 2^-25 of the largest.  The weighted sum of L
  values accumulates L / 16 + 64 roundings.  The bound below takes
  2 ds (numerator and denominator) times sum p|v|, which holds every element.
"""
import math

import torch

U16, U32 = 2.0 ** -11, 2.0 ** -24


def transform(x, w, eps, positions, inv_freq, pairs, mag):
    """(y, pair size): norm and rotation of [T, H, D] heads in fp64."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    y, size = x.clone(), x.abs()
    if inv_freq is not None:
        R = 2 * inv_freq.numel()
        ang = positions.double()[:, None, None] * inv_freq.double()
        c, s = torch.cos(ang) * mag, torch.sin(ang) * mag
        ia = torch.arange(0, R, 2, device=x.device) if pairs else torch.arange(R // 2, device=x.device)
        ib = ia + 1 if pairs else ia + R // 2
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = size[..., ib] = (a.abs() + b.abs()) * abs(mag)
    return y, size


def assert_transform(got, want, size, what=""):
    err = (got.double() - want).abs()
    bound = 32 * U32 * size
    if got.dtype == torch.float16:
        bound = bound + U16 * want.abs() + 2.0 ** -25
    else:
        bound = bound + U32 * want.abs()
    assert torch.isfinite(got).all(), what
    assert (err <= bound).all(), f"{what}: worst error / bound {(err / bound.clamp_min(1e-300)).max().item():.3f}"


def attention(q, k, v, base, causal, window, scale):
    """q [n, Hq, D] of tokens at cache indexes base .. base + n - 1 over k, v
    [L, Hkv, D]: (y, lse, bound of |y| errors before the output rounding, bound of lse errors)."""
    n, Hq, D = q.shape
    L, Hkv = k.shape[:2]
    G = Hq // Hkv
    i = base + torch.arange(n, device=q.device)[:, None]
    j = torch.arange(L, device=q.device)[None, :]
    seen = torch.ones((n, L), dtype=torch.bool, device=q.device)
    if causal:
        seen &= j <= i
    if window:
        seen &= j > i - window
    seen &= (i >= 0)
    y = torch.zeros((n, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    by, bl = torch.zeros_like(y), torch.zeros_like(lse)
    any_seen = seen.any(1)
    if L == 0 or not any_seen.any():
        return y, lse, by, bl
    needed = seen.any(0)
    kd = torch.where(needed[:, None, None], k, torch.zeros_like(k)).double()
    vd = torch.where(needed[:, None, None], v, torch.zeros_like(v)).double()
    for h in range(Hq):
        kh, vh = kd[:, h // G], vd[:, h // G]
        s = q[:, h].double() @ kh.T * scale
        s = torch.where(seen, s, torch.full_like(s, -math.inf))
        m = s.amax(1, keepdim=True)
        m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
        p = torch.exp(s - m)
        l = p.sum(1, keepdim=True)
        live = l[:, 0] > 0
        inv = torch.where(l > 0, 1 / l, torch.zeros_like(l))
        y[:, h] = (p @ vh) * inv
        lse[:, h] = torch.where(live, (m + torch.log(l))[:, 0], torch.full_like(l[:, 0], -math.inf))
        A = (p @ vh.abs()) * inv
        dot = torch.where(seen, q[:, h].double().abs() @ kh.abs().T, torch.zeros_like(s)).amax(1)
        top = torch.where(seen, s, torch.zeros_like(s)).abs().amax(1)
        ds = scale * (D + 2) * U32 * dot + 4 * U32 * top + 2.0 ** -20
        by[:, h] = (2 * ds[:, None] + U16 + (L / 16 + 64) * U32) * A + \
            L * 2.0 ** -25 * vh.abs().amax() * inv
        bl[:, h] = 2 * ds + (L / 16 + 64) * U32 + 2.0 ** -22 * torch.where(live, lse[:, h].abs(), top)
    return y, lse, by, bl


def paged(lens, page, Hkv, D, order, gen, first=None, spare=3, device="cuda", interleaved=False):
    """A cache of shuffled pages with keys and values of lens[b] tokens from first[b] on;
    every other place is NaN or infinite and every other table entry -1.
    Returns k, v as [pages, page, Hkv, D] views, the table and the dense per-sequence k, v."""
    need = [(L + page - 1) // page for L in lens]
    total = sum(need) + spare
    shape = (total, page, Hkv, D) if order == "tokens" else (total, Hkv, page, D)
    junk = torch.tensor([math.nan, math.inf, -math.inf, math.nan], dtype=torch.float16, device=device)
    fill = lambda: junk[torch.randint(0, 4, shape, generator=gen, device=device)]
    if interleaved:
        both = torch.stack([fill(), fill()], 1)
        k, v = both[:, 0], both[:, 1]
    else:
        k, v = fill(), fill()
    if order == "heads":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    perm = torch.randperm(total, generator=gen, device=device).to(torch.int32)
    table = torch.full((len(lens), max(need + [0]) + 2), -1, dtype=torch.int32, device=device)
    dense, at = [], 0
    for b, L in enumerate(lens):
        f = first[b] if first else 0
        table[b, f // page:need[b]] = perm[at + f // page:at + need[b]]
        kd = torch.full((L, Hkv, D), math.nan, dtype=torch.float16, device=device)
        vd = kd.clone()
        if L > f:
            kd[f:] = torch.randn((L - f, Hkv, D), generator=gen, device=device).half()
            vd[f:] = torch.randn((L - f, Hkv, D), generator=gen, device=device).half()
            p = torch.arange(f, L, device=device)
            ids = table[b].long()[p // page]
            k[ids, p % page], v[ids, p % page] = kd[f:], vd[f:]
        dense.append((kd, vd))
        at += need[b]
    return k, v, table, dense
