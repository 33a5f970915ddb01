"""Work cases of the attention operators that stand between the quantized
linears of a decoder layer:

* ``rope``    -- exl3_qk_norm_rope: the RMS norm of every query and key head
                 and the rotary position rotation, in one pass;
* ``append``  -- exl3_qkv_append: the same, with the keys and values written
                 to their places in a paged cache;
* ``attend``  -- exl3_paged_attention: attention of each sequence's new tokens
                 (one, a few or a whole chunk) over its paged cache.

A case is a dict of plain values.  ``prepare(case, seed)`` makes the inputs on
the GPU, ``run(state)`` makes one pass: with ``own`` false from elementary
torch operations in 32 bits (angles in 64), with ``own`` true through the
library's entry points.  ``exact(case, seed)`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

# Head counts and sizes: 40 query and 8 key/value heads of 128 are the widths
# 5120 + 1024 + 1024 of the fused q, k, v shards over k = 5120; 16 and 2 heads
# of 256 with a quarter of the head rotated go with the hidden size 2048 of
# the routed-expert workload; 64-wide heads are the smallest size served.


def listed():
    return [
        # one decode step of one user: latency of the smallest call
        dict(name="rope_step", op="rope", T=1, Hq=40, Hkv=8, D=128, R=128, layout="half", norm=True, fp32=False,
             far=4096, scaling="none"),
        # a prefill chunk at far positions of a long-context model, a quarter of each head rotated
        dict(name="rope_chunk_far", op="rope", T=4096, Hq=16, Hkv=2, D=256, R=64, layout="half", norm=True,
             fp32=False, far=1000000, scaling="yarn"),
        # an odd chunk of fp32 projections, neighbouring pairs rotated, no norms
        dict(name="rope_odd_pairs", op="rope", T=1777, Hq=24, Hkv=8, D=64, R=64, layout="pairs", norm=False,
             fp32=True, far=30000, scaling="bands"),
        # a decode step of 32 users, each token to its own page of 16
        dict(name="append_step_32", op="append", B=32, new=1, old=4000, Hq=40, Hkv=8, D=128, R=128, layout="half",
             norm=True, fp32=False, page=16, order="tokens", scaling="none"),
        # prefill of four ragged prompts at once
        dict(name="append_prompts", op="append", B=4, new=3000, old=0, Hq=40, Hkv=8, D=128, R=128, layout="half",
             norm=True, fp32=False, page=64, order="tokens", scaling="none"),
        # ragged chunks behind long histories: fp32 projections, pages of 48 tokens, a head's tokens adjacent
        dict(name="append_chunks_d256", op="append", B=3, new=700, old=30000, Hq=16, Hkv=2, D=256, R=64,
             layout="half", norm=True, fp32=True, page=48, order="heads", scaling="yarn"),
        # one user, a short history: latency
        dict(name="attend_step_short", op="attend", B=1, new=1, old=500, ragged=False, Hq=40, Hkv=8, D=128, page=16,
             order="tokens", window=0),
        # one user, a very long history: the cache has to be split over all SMs
        dict(name="attend_step_long", op="attend", B=1, new=1, old=131000, ragged=False, Hq=40, Hkv=8, D=128, page=64,
             order="tokens", window=0),
        # 64 users with histories of very different lengths
        dict(name="attend_step_64", op="attend", B=64, new=1, old=8000, ragged=True, Hq=40, Hkv=8, D=128, page=16,
             order="tokens", window=0),
        # a few drafted tokens per user to be verified, 8 query heads to a key head of 256
        dict(name="attend_verify_d256", op="attend", B=8, new=5, old=20000, ragged=True, Hq=16, Hkv=2, D=256, page=32,
             order="heads", window=0),
        # a whole prompt
        dict(name="attend_prompt", op="attend", B=1, new=8192, old=0, ragged=False, Hq=40, Hkv=8, D=128, page=64,
             order="tokens", window=0),
        # a chunk of a long prompt
        dict(name="attend_chunk_d256", op="attend", B=1, new=2047, old=63000, ragged=False, Hq=16, Hkv=2, D=256,
             page=128, order="heads", window=0),
    ]


def _logint(rng, lo, hi):
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
    return max(lo, min(hi, v))


def _heads(rng):
    return rng.choice([(40, 8, 128), (16, 2, 256), (24, 8, 64), (8, 8, 128), (32, 4, 128), (12, 4, 64), (16, 8, 256),
                       (7, 1, 128)])


def draw(rng):
    """One more case of the listed cases' ranges."""
    op = rng.choice(["rope", "append", "attend", "attend"])
    Hq, Hkv, D = _heads(rng)
    rot = dict(R=rng.choice([D, D, D // 2, D // 4]), layout=rng.choice(["half", "pairs"]), norm=rng.random() < 0.6,
               fp32=rng.random() < 0.4, scaling=rng.choice(["none", "linear", "ntk", "bands", "yarn"]))
    if op == "rope":
        return dict(op=op, T=_logint(rng, 1, 4096 * 4608 // ((Hq + Hkv) * D)), Hq=Hq, Hkv=Hkv, D=D,
                    far=_logint(rng, 64, 1000000), **rot)
    page = rng.choice([16, 32, 48, 64, 128, 256])
    order = rng.choice(["tokens", "heads"])
    if op == "append":
        B = _logint(rng, 1, 64)
        return dict(op=op, B=B, new=_logint(rng, 1, max(1, 5000 // B)), old=_logint(rng, 1, 30000 // B + 1) - 1,
                    Hq=Hq, Hkv=Hkv, D=D, page=page, order=order, **rot)
    kind = rng.choice(["step", "few", "chunk"])
    new = 1 if kind == "step" else rng.randint(2, 16) if kind == "few" else _logint(rng, 17, 4096)
    B = _logint(rng, 1, 64) if kind != "chunk" else _logint(rng, 1, 4)
    # the largest listed cases read 0.6 to 1.2 GB of cache and form 2.7e9 scores
    longest = min(131000, 1_000_000_000 // (B * Hkv * D * 4), 2_000_000_000 // (B * new * Hq))
    old = _logint(rng, 1, max(1, longest - new)) - 1
    window = rng.choice([0, 0, _logint(rng, 1, 8192)])
    return dict(op=op, B=B, new=new, old=old, ragged=rng.random() < 0.6, Hq=Hq, Hkv=Hkv, D=D, page=page, order=order,
                window=window)


# ------------------------------------------------------------------ lengths

def _lengths(case):
    """(new tokens, tokens behind them) of each sequence."""
    B, new, old = case["B"], case["new"], case["old"]
    r = random.Random(B * 1000003 + new * 1009 + old)
    out = []
    for b in range(B):
        if B > 1 and case.get("ragged", True):
            n = new if new <= 16 else r.randint(max(1, new // 2), new)
            o = int(old * r.random() ** 2) if b else old
        else:
            n, o = new, old
        out.append((n, o))
    return out


def _frequencies(case):
    """Rotary frequencies and the rotation's magnitude for the case's scaling,
    computed in 64 bits and rounded to fp32, as a model's set-up does."""
    R = case["R"]
    base, factor, orig, low, high = 10000.0, 8.0, 4096.0, 1.0, 4.0
    mag = 1.0
    i = torch.arange(0, R, 2, dtype=torch.float64)
    if case["scaling"] == "ntk":
        base = base * factor ** (R / (R - 2))
    f = base ** (-i / R)
    turns = orig * f / (2 * math.pi)                 # rotations within the original context
    if case["scaling"] == "linear":
        f = f / factor
    elif case["scaling"] == "bands":
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        f = f / factor * (1 - keep) + f * keep
    elif case["scaling"] == "yarn":
        low, high = 1.0, 32.0
        place = lambda n: R * math.log(orig / (n * 2 * math.pi)) / (2 * math.log(base))
        first, last = max(0, math.floor(place(high))), min(R - 1, math.ceil(place(low)))
        keep = 1 - ((torch.arange(R // 2, dtype=torch.float64) - first) / max(last - first, 0.001)).clamp(0, 1)
        f = f / factor * (1 - keep) + f * keep
        mag = 0.1 * math.log(factor) + 1.0
    return f.to(torch.float32), mag


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _pages(case, lens, g):
    """A cache of shuffled pages and its page table (entries past a
    sequence's end are -1, as an allocator leaves them)."""
    page, Hkv, D = case["page"], case["Hkv"], case["D"]
    need = [(n + o + page - 1) // page for n, o in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need) + 2), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    shape = (total, page, Hkv, D) if case["order"] == "tokens" else (total, Hkv, page, D)
    k = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)
    if case["order"] == "heads":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    return k, v, table                               # [pages, page, Hkv, D] views


def _batch(lens):
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    kv_len = torch.tensor([n + o for n, o in lens], dtype=torch.int32, device="cuda")
    return q_start, kv_len


def prepare(case, seed):
    g = _gen(seed)
    op, Hq, Hkv, D = case["op"], case["Hq"], case["Hkv"], case["D"]
    s = dict(case=dict(case))
    if op in ("rope", "append"):
        lens = _lengths(case) if op == "append" else None
        T = case["T"] if op == "rope" else sum(n for n, _ in lens)
        dt = torch.float32 if case["fp32"] else torch.float16
        # projections of outlier channels: most values near one, some channels far larger
        ch = torch.exp(0.7 * torch.randn((Hq + Hkv, D), generator=g, device="cuda"))
        qk = torch.randn((T, Hq + Hkv, D), generator=g, device="cuda") * ch
        s["q"], s["k"] = qk[:, :Hq].contiguous().to(dt), qk[:, Hq:].contiguous().to(dt)
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            w = (1 + 0.3 * torch.randn((2, D), generator=g, device="cuda")).to(torch.float16)
            s["q_norm"], s["k_norm"] = w[0].contiguous(), w[1].contiguous()
        f, s["mag"] = _frequencies(case)
        s["inv_freq"] = f.cuda()
        if op == "rope":
            start = int(torch.randint(0, max(1, case["far"] - T), (1,), generator=g, device="cuda"))
            s["positions"] = torch.arange(start, start + T, dtype=torch.int32, device="cuda")
        else:
            s["v"] = torch.randn((T, Hkv, D), generator=g, device="cuda").to(dt)
            s["k_cache"], s["v_cache"], s["table"] = _pages(case, lens, g)
            s["q_start"], s["kv_len"] = _batch(lens)
        s["q_out"] = torch.empty((T, Hq, D), dtype=torch.float16, device="cuda")
        s["k_out"] = torch.empty((T, Hkv, D), dtype=torch.float16, device="cuda") if op == "rope" else None
    else:
        lens = _lengths(case)
        T = sum(n for n, _ in lens)
        s["k_cache"], s["v_cache"], s["table"] = _pages(case, lens, g)
        s["q_start"], s["kv_len"] = _batch(lens)
        # scores of a standard deviation of two: some keys stand out
        s["q"] = (2 * torch.randn((T, Hq, D), generator=g, device="cuda")).to(torch.float16)
        s["y"] = torch.empty((T, Hq, D), dtype=torch.float16, device="cuda")
        s["lse"] = torch.empty((T, Hq), dtype=torch.float32, device="cuda")
    s["lens"] = lens
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program keeps beside its tensors: the library's descriptors."""
    if "tq" not in s:
        import trellis_quantized_gb300 as tq
        s["tq"] = tq
        if "inv_freq" in s:
            layout = tq.EXL3_ROPE_HALF if s["case"]["layout"] == "half" else tq.EXL3_ROPE_PAIRS
            s["ht"] = tq.head_transform(q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6, inv_freq=s["inv_freq"],
                                        layout=layout, magnitude=s["mag"])
        if "table" in s:
            s["cache"] = tq.kv_cache(s["k_cache"], s["v_cache"])
            s["batch"] = tq.paged_batch(s["q_start"], s["kv_len"], s["table"])
    return s["tq"]


# -------------------------------------------------------------- plain forms

def _transform(x, w, positions, inv_freq, R, layout, mag):
    """Norm and rotation of [T, H, D] heads in fp32 (angles in fp64)."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    ang = positions.double()[:, None] * inv_freq.double()[None, :]
    c = (torch.cos(ang) * mag).float()[:, None, :]
    sn = (torch.sin(ang) * mag).float()[:, None, :]
    out = x.clone()
    if layout == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        out[..., :R // 2] = a * c - b * sn
        out[..., R // 2:R] = b * c + a * sn
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        out[..., 0:R:2] = a * c - b * sn
        out[..., 1:R:2] = b * c + a * sn
    return out


def _positions(s):
    """Position of every new token and its place (page, offset) in the cache."""
    pos, seq = [], []
    for b, (n, o) in enumerate(s["lens"]):
        pos.append(torch.arange(o, o + n, device="cuda"))
        seq.append(torch.full((n,), b, dtype=torch.int64, device="cuda"))
    pos, seq = torch.cat(pos), torch.cat(seq)
    page = s["case"]["page"]
    return pos, s["table"][seq, pos // page].long(), pos % page


def _gather(s, b, L):
    """Keys and values 0 .. L-1 of sequence b, [L, Hkv, D] fp16."""
    page = s["case"]["page"]
    ids = s["table"][b, :(L + page - 1) // page].long()
    shape = (-1, s["case"]["Hkv"], s["case"]["D"])
    return s["k_cache"][ids].reshape(shape)[:L], s["v_cache"][ids].reshape(shape)[:L]


def _attend(s, dtype, rows_at_once):
    """Attention in `dtype`: (y, lse), one head group at a time."""
    case = s["case"]
    Hq, Hkv, D, window = case["Hq"], case["Hkv"], case["D"], case["window"]
    G, scale = Hq // Hkv, 1.0 / math.sqrt(D)
    T = s["q"].shape[0]
    y = torch.empty((T, Hq, D), dtype=dtype, device="cuda")
    lse = torch.empty((T, Hq), dtype=dtype, device="cuda")
    t = 0
    for b, (n, o) in enumerate(s["lens"]):
        L = n + o
        k, v = _gather(s, b, L)
        for r in range(0, n, rows_at_once):
            m = min(rows_at_once, n - r)
            first = max(0, o + r - window + 1) if window else 0
            last = o + r + m
            i = torch.arange(o + r, last, device="cuda")[:, None]
            j = torch.arange(first, last, device="cuda")[None, :]
            hide = j > i
            if window:
                hide = hide | (j <= i - window)
            group = Hkv if m * Hq * (last - first) <= (1 << 26) else 1     # kv heads in one product
            for h in range(0, Hkv, group):
                kk = k[first:last, h:h + group].to(dtype).permute(1, 2, 0)            # [g, D, keys]
                vv = v[first:last, h:h + group].to(dtype).permute(1, 0, 2)            # [g, keys, D]
                q = s["q"][t + r:t + r + m, h * G:(h + group) * G].to(dtype)
                q = q.view(m, group, G, D).permute(1, 2, 0, 3).reshape(group, G * m, D)
                sc = torch.matmul(q, kk).view(group, G, m, last - first) * scale
                sc.masked_fill_(hide, float("-inf"))
                top = sc.amax(-1, keepdim=True)
                sc = sc.sub_(top).exp_()
                tot = sc.sum(-1, keepdim=True)
                o_ = torch.matmul(sc.view(group, G * m, -1), vv).view(group, G, m, D) / tot
                y[t + r:t + r + m, h * G:(h + group) * G] = o_.permute(2, 0, 1, 3).reshape(m, group * G, D)
                ls = (top + tot.log()).squeeze(-1)
                lse[t + r:t + r + m, h * G:(h + group) * G] = ls.permute(2, 0, 1).reshape(m, group * G)
        t += n
    return y, lse


def _plain(s):
    case = s["case"]
    if case["op"] == "attend":
        y, lse = _attend(s, torch.float32, 2048)
        return dict(y=y.to(torch.float16), lse=lse)
    R, layout, mag = case["R"], case["layout"], s["mag"]
    if case["op"] == "rope":
        f = lambda x, w: _transform(x, w, s["positions"], s["inv_freq"], R, layout, mag).to(torch.float16)
        return dict(q=f(s["q"], s["q_norm"]), k=f(s["k"], s["k_norm"]))
    pos, page, off = _positions(s)
    f = lambda x, w: _transform(x, w, pos, s["inv_freq"], R, layout, mag).to(torch.float16)
    q = f(s["q"], s["q_norm"])
    s["k_cache"][page, off] = f(s["k"], s["k_norm"])
    s["v_cache"][page, off] = s["v"].to(torch.float16)
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def run(state):
    if not own:
        return _plain(state)
    s = state
    tq = _handles(s)
    op = s["case"]["op"]
    if op == "rope":
        tq.exl3_qk_norm_rope(s["q"], s["k"], s["positions"], s["ht"], q_out=s["q_out"], k_out=s["k_out"])
        return dict(q=s["q_out"], k=s["k_out"])
    if op == "append":
        tq.exl3_qkv_append(s["q"], s["k"], s["v"], s["batch"], s["cache"], s["ht"], q_out=s["q_out"])
        return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])
    tq.exl3_paged_attention(s["q"], s["batch"], s["cache"], window=s["case"]["window"], y=s["y"], lse=s["lse"])
    return dict(y=s["y"], lse=s["lse"])


# ---------------------------------------------------------------- definition

def _exact_heads(x, w, positions, inv_freq, R, layout, mag):
    """Each pair (a, b) as the complex number a + ib, turned by its angle."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * w.double()
    turn = torch.polar(torch.full((positions.numel(), R // 2), float(mag), dtype=torch.float64, device="cuda"),
                       positions.double().outer(inv_freq.double()))
    rot, rest = x[..., :R], x[..., R:]
    pairs = rot.unflatten(-1, (2, R // 2)).transpose(-1, -2) if layout == "half" else rot.unflatten(-1, (R // 2, 2))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None, :])
    rot = z.transpose(-1, -2).flatten(-2) if layout == "half" else z.flatten(-2)
    return torch.cat([rot, rest], -1)


def _exact_attend(s):
    """Softmax-weighted means in 64 bits, one query head and one slice of rows at a time."""
    case = s["case"]
    Hq, G, D, W = case["Hq"], case["Hq"] // case["Hkv"], case["D"], case["window"]
    y = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, o) in enumerate(s["lens"]):
        p = torch.arange(n + o, device="cuda")
        ids = s["table"][b].long()[p // case["page"]]
        for h in range(case["Hkv"]):
            k = s["k_cache"][ids, p % case["page"], h].double()
            v = s["v_cache"][ids, p % case["page"], h].double()
            for r in range(0, n, 512):
                e = min(n, r + 512)
                lo, hi = max(0, o + r + 1 - W) if W else 0, o + e
                q = s["q"][t0 + r:t0 + e, h * G:(h + 1) * G].double()
                z = torch.einsum("tgd,jd->gtj", q, k[lo:hi]) / math.sqrt(D)
                dist = (o + torch.arange(r, e, device="cuda"))[:, None] - p[lo:hi][None, :]
                seen = (dist >= 0) & (dist < W) if W else dist >= 0
                z = torch.where(seen, z, torch.full_like(z, float("-inf")))
                ls = torch.logsumexp(z, -1)
                prob = torch.exp(z - ls[..., None])
                y[t0 + r:t0 + e, h * G:(h + 1) * G] = torch.einsum("gtj,jd->tgd", prob, v[lo:hi])
                lse[t0 + r:t0 + e, h * G:(h + 1) * G] = ls.T
        t0 += n
    return y, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        if _scores(case) * case["Hq"] * case["D"] > 2.5e12:
            return None
        y, lse = _exact_attend(s)
        return dict(y=y, lse=lse)
    args = (s["inv_freq"], case["R"], case["layout"], s["mag"])
    if case["op"] == "rope":
        return dict(q=_exact_heads(s["q"], s["q_norm"], s["positions"], *args),
                    k=_exact_heads(s["k"], s["k_norm"], s["positions"], *args))
    pos = torch.cat([torch.arange(o, o + n, device="cuda") for n, o in s["lens"]])
    q = _exact_heads(s["q"], s["q_norm"], pos, *args)
    k = _exact_heads(s["k"], s["k_norm"], pos, *args)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    t = 0
    for b, (n, o) in enumerate(s["lens"]):
        row = s["table"][b].cpu().tolist()
        for first in range(o - o % case["page"], o + n, case["page"]):
            lo, hi = max(first, o), min(first + case["page"], o + n)
            pg = row[first // case["page"]]
            kc[pg, lo - first:hi - first] = k[t + lo - o:t + hi - o]
            vc[pg, lo - first:hi - first] = s["v"][t + lo - o:t + hi - o].double()
        t += n
    return dict(q=q, k_cache=kc, v_cache=vc)


# ---------------------------------------------------------------------- work

def _scores(case):
    """Query-key pairs of one query head."""
    W, total = case["window"], 0
    for n, o in _lengths(case):
        if W:
            total += sum(min(W, o + i + 1) for i in range(n))
        else:
            total += n * o + n * (n + 1) // 2
    return total


def work(case):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "attend":
        lens, W = _lengths(case), case["window"]
        T = sum(n for n, _ in lens)
        keys = sum(min(n + o, n + W - 1) if W else n + o for n, o in lens)
        tables = sum((n + o + case["page"] - 1) // case["page"] for n, o in lens)
        return dict(bytes=keys * Hkv * D * 4 + T * Hq * (D * 4 + 4) + tables * 4 + 8 * len(lens),
                    flops=4 * D * Hq * _scores(case))
    T = case["T"] if case["op"] == "rope" else sum(n for n, _ in _lengths(case))
    size = 4 if case["fp32"] else 2
    heads = Hq + Hkv + (Hkv if case["op"] == "append" else 0)
    elems = T * (Hq + Hkv) * D
    return dict(bytes=T * heads * D * (size + 2) + (T * 4 if case["op"] == "rope" else 8 * case["B"]) + case["R"] * 2,
                flops=elems * ((4 if case["norm"] else 0) + 3))
