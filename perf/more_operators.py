"""Work cases of the operators that follow a token's own choices beside the
quantized weights -- which experts it takes, which request's adapter applies:

* ``logits``  -- exl3_router_logits: the router's product, hidden states
                 against one row of weights per expert, with fp16 weights as
                 they are or fp32 weights kept to 22 bits and more;
* ``route``   -- exl3_route: expert ids and weights from the logits (softmax
                 or sigmoid scores, a balance bias, groups, top-k), as
                 exl3_moe_grouped takes them;
* ``adapt``   -- exl3_adapter_add: low-rank adapters of many requests at once
                 added to a linear's output.

A case is a dict of plain values.  ``prepare(case, seed)`` makes the inputs on
the GPU, ``run(state)`` makes one pass: with ``own`` false from elementary
torch operations in 32 bits (selection values in 64), with ``own`` true
through the library's entry points.  ``exact(case, seed)`` is the definition
in 64 bits.
"""
import math
import random

import torch

own = False

# Hidden size 2048 with 256 experts and top 8 is the routed-expert workload of
# the benchmark; 5120 -> 5120 / 17408 and 4096 -> 4096 are its dense linears.


def listed():
    return [
        # one decode step of one user: the smallest call, latency
        dict(name="logits_step", op="logits", T=1, k=2048, E=256, fp32=False, bias=False),
        # a decode step of 48 users; the router's weights are kept in fp32
        dict(name="logits_users", op="logits", T=48, k=2048, E=256, fp32=True, bias=False),
        # a prefill chunk of the benchmark's routed-expert layer
        dict(name="logits_chunk", op="logits", T=4096, k=2048, E=256, fp32=False, bias=False),
        # an odd chunk, an odd number of experts, fp32 weights and a bias
        dict(name="logits_odd", op="logits", T=1333, k=5120, E=60, fp32=True, bias=True),
        # routing of one token: latency
        dict(name="route_step", op="route", T=1, E=256, topk=8, score="softmax", bias=False, groups=1, kept=1,
             group="max", renorm=True, scale=1.0, fp16=False),
        # a prefill chunk, softmax over the chosen eight
        dict(name="route_chunk", op="route", T=4096, E=256, topk=8, score="softmax", bias=False, groups=1, kept=1,
             group="max", renorm=True, scale=1.0, fp16=False),
        # sigmoid scores with a balance bias, four of eight groups by their two best experts
        dict(name="route_groups", op="route", T=2500, E=256, topk=8, score="sigmoid", bias=True, groups=8, kept=4,
             group="top2", renorm=True, scale=2.5, fp16=False),
        # few experts, an odd number of them, scores of the whole softmax, fp16 logits of a quantized router
        dict(name="route_odd", op="route", T=777, E=60, topk=4, score="softmax", bias=False, groups=1, kept=1,
             group="max", renorm=False, scale=1.0, fp16=True),
        # one token with its adapter: latency
        dict(name="adapt_step", op="adapt", B=1, new=1, chunks=0, N=8, share=1, rank=16, ranks=False, k=5120, n=5120,
             none=False, fp32=False),
        # a decode step of 64 users on two dozen adapters of different ranks, some users without one
        dict(name="adapt_users", op="adapt", B=64, new=1, chunks=0, N=24, share=2, rank=64, ranks=True, k=5120,
             n=17408, none=True, fp32=False),
        # ragged prompts, each with its own small adapter, beside the widest linear but one
        dict(name="adapt_prompts", op="adapt", B=4, new=2000, chunks=4, N=8, share=1, rank=16, ranks=False, k=5120,
             n=17408, none=False, fp32=False),
        # a prompt's chunk among decode steps, large ranks, fp32 output
        dict(name="adapt_mixed", op="adapt", B=41, new=2000, chunks=1, N=16, share=3, rank=128, ranks=True, k=4096,
             n=4096, none=True, fp32=True),
    ]


def _logint(rng, lo, hi):
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
    return max(lo, min(hi, v))


def draw(rng):
    """One more case of the listed cases' ranges."""
    op = rng.choice(["logits", "route", "adapt"])
    if op == "logits":
        k = rng.choice([1024, 2048, 4096, 5120, 128 * rng.randint(4, 56)])
        E = rng.choice([8, 32, 60, 64, 128, 256, rng.randint(4, 512)])
        return dict(op=op, T=_logint(rng, 1, min(8192, 4096 * 2048 * 256 // (k * E))), k=k, E=E,
                    fp32=rng.random() < 0.4, bias=rng.random() < 0.3)
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * rng.choice([8, 16, 20, 32, 64, rng.randint(4, 64)])
        kept = rng.randint(1, groups)
        return dict(op=op, T=_logint(rng, 1, min(8192, 4096 * 256 // E)), E=E, topk=rng.randint(1, min(12, E // groups * kept)),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, kept=kept,
                    group=rng.choice(["max", "top2"]), renorm=rng.random() < 0.7, scale=rng.choice([1.0, 1.0, 2.5]),
                    fp16=rng.random() < 0.3)
    k, n = (rng.choice([512, 2048, 4096, 5120, 17408, 128 * rng.randint(2, 60)]) for _ in range(2))
    rank = rng.choice([8, 16, 16, 32, 64, 128])
    kind = rng.choice(["steps", "steps", "prompts", "mixed"])
    B = _logint(rng, 1, 256) if kind == "steps" else _logint(rng, 1, 8) if kind == "prompts" else _logint(rng, 2, 96)
    new = 1 if kind == "steps" and rng.random() < 0.7 else rng.randint(2, 6) if kind == "steps" else \
        _logint(rng, 20, max(21, min(4096, 6000 * 22000 // (k + 2 * n) // min(B, 8))))
    chunks = 0 if kind == "steps" else B if kind == "prompts" else max(1, B // 16)
    return dict(op=op, B=B, new=new, chunks=chunks, N=_logint(rng, 1, 48), share=rng.randint(1, 4), rank=rank,
                ranks=rng.random() < 0.4, k=k, n=n, none=rng.random() < 0.4, fp32=rng.random() < 0.3)


# ------------------------------------------------------------------ batches

def _sequences(case):
    """(rows, adapter) of each sequence, -1 for none, and each adapter's rank."""
    B, N = case["B"], case["N"]
    r = random.Random(B * 1000003 + N * 1009 + case["new"])
    live = max(1, min(N, B // case["share"]))        # the adapters in use; users share them
    ids = r.sample(range(N), live)
    seqs = []
    for b in range(B):
        if b < case["chunks"]:
            rows = r.randint(max(1, case["new"] // 2), case["new"])
        else:
            rows = case["new"] if not case["chunks"] else 1
        a = -1 if case["none"] and b and r.random() < 0.2 else ids[b % live]
        seqs.append((rows, a))
    r.shuffle(seqs)
    R = case["rank"]
    ranks = [r.choice([x for x in (8, 16, 32, 64, 128) if x <= R]) if case["ranks"] else R for _ in range(N)]
    return seqs, ranks


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _hidden(T, k, g):
    """Hidden states near one with a few channels thirty times as large."""
    x = torch.randn((T, k), generator=g, device="cuda")
    x *= torch.where(torch.rand(k, generator=g, device="cuda") < 0.005, 30.0, 1.0)
    return x.to(torch.float16)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=dict(case))
    if op == "logits":
        T, k, E = case["T"], case["k"], case["E"]
        s["x"] = _hidden(T, k, g)
        w = torch.randn((E, k), generator=g, device="cuda") / math.sqrt(k)
        s["w"] = w if case["fp32"] else w.to(torch.float16)
        s["bias"] = torch.randn(E, generator=g, device="cuda") if case["bias"] else None
        s["logits"] = torch.empty((T, E), dtype=torch.float32, device="cuda")
    elif op == "route":
        T, E, topk = case["T"], case["E"], case["topk"]
        l = torch.randn((T, E), generator=g, device="cuda") * 1.5
        s["logits"] = l.to(torch.float16) if case["fp16"] else l
        s["bias"] = 0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
        s["ids"] = torch.empty((T, topk), dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty((T, topk), dtype=torch.float32, device="cuda")
    else:
        seqs, ranks = _sequences(case)
        N, R, k, n = case["N"], case["rank"], case["k"], case["n"]
        T = sum(rows for rows, _ in seqs)
        s["seqs"], s["ranks"] = seqs, ranks
        s["x"] = _hidden(T, k, g)
        s["a"] = (torch.randn((N, R, k), generator=g, device="cuda") / math.sqrt(k)).to(torch.float16)
        s["b"] = (torch.randn((N, n, R), generator=g, device="cuda") / math.sqrt(R)).to(torch.float16)
        for a, r in enumerate(ranks):                # a slot holds zeros past its adapter's rank
            s["a"][a, r:] = 0
            s["b"][a, :, r:] = 0
        s["scale"] = torch.rand(N, generator=g, device="cuda") + 0.5
        s["rank"] = torch.tensor(ranks, dtype=torch.int32, device="cuda")
        dt = torch.float32 if case["fp32"] else torch.float16
        s["y"] = torch.randn((T, n), generator=g, device="cuda").to(dt)
        s["out"] = torch.empty((T, n), dtype=dt, device="cuda")
        starts = [0]
        for rows, _ in seqs:
            starts.append(starts[-1] + rows)
        s["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["ids"] = torch.tensor([a for _, a in seqs], dtype=torch.int32, device="cuda")
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program keeps beside its tensors: the router's packed weights,
    the routing rule, the adapters' descriptor, and the step's adapter plan,
    which serves every linear of every layer."""
    if "tq" not in s:
        import trellis_quantized_gb300 as tq
        s["tq"] = tq
        case = s["case"]
        if case["op"] == "logits":
            s["router"] = tq.router(s["w"], bias=s["bias"])
        elif case["op"] == "route":
            s["rule"] = tq.route_rule(
                case["topk"], score=tq.EXL3_SCORE_SOFTMAX if case["score"] == "softmax" else tq.EXL3_SCORE_SIGMOID,
                bias=s["bias"], groups=case["groups"], groups_kept=case["kept"],
                group_score=tq.EXL3_GROUP_MAX if case["group"] == "max" else tq.EXL3_GROUP_TOP2,
                renormalise=case["renorm"], scale=case["scale"])
        else:
            s["adapters"] = tq.adapters(s["a"], s["b"], s["scale"], rank=s["rank"] if case["ranks"] else None)
            s["plan"] = tq.exl3_adapter_plan(s["q_start"], s["ids"], s["x"].shape[0], case["N"])
    return s["tq"]


# -------------------------------------------------------------- plain forms

def _plain_route(s):
    case = s["case"]
    logits, T, E = s["logits"], case["T"], case["E"]
    l = logits.double()
    if case["score"] == "softmax":
        p = (l - l.amax(-1, keepdim=True)).exp()
        p = p / p.sum(-1, keepdim=True)
    else:
        p = 1 / (1 + (-l).exp())
    c = p + s["bias"].double() if s["bias"] is not None else p
    if case["groups"] > 1:
        in_group = c.view(T, case["groups"], -1).sort(dim=-1, descending=True).values
        best = in_group[..., 0] if case["group"] == "max" else in_group[..., :2].sum(-1)
        order = best.sort(dim=-1, descending=True, stable=True).indices[:, :case["kept"]]
        keep = torch.zeros((T, case["groups"]), dtype=torch.bool, device="cuda").scatter_(1, order, True)
        c = c.masked_fill(~keep.repeat_interleave(E // case["groups"], 1), float("-inf"))
    ids = c.sort(dim=-1, descending=True, stable=True).indices[:, :case["topk"]]
    w = p.float().gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return dict(ids=ids.to(torch.int32), weights=w * case["scale"])


def _plain(s):
    case = s["case"]
    if case["op"] == "logits":
        y = torch.matmul(s["x"].float(), s["w"].float().t())
        return dict(logits=y + s["bias"] if s["bias"] is not None else y)
    if case["op"] == "route":
        return _plain_route(s)
    out = torch.empty_like(s["y"])
    t = 0
    for rows, a in s["seqs"]:
        y = s["y"][t:t + rows].float()
        if a >= 0:
            h = torch.matmul(s["x"][t:t + rows].float(), s["a"][a].float().t())
            y = y + s["scale"][a] * torch.matmul(h, s["b"][a].float().t())
        out[t:t + rows] = y.to(out.dtype)
        t += rows
    return dict(out=out)


def run(state):
    if not own:
        return _plain(state)
    s = state
    tq = _handles(s)
    op = s["case"]["op"]
    if op == "logits":
        tq.exl3_router_logits(s["x"], s["router"], logits=s["logits"])
        return dict(logits=s["logits"])
    if op == "route":
        tq.exl3_route(s["logits"], s["rule"], ids=s["ids"], weights=s["weights"])
        return dict(ids=s["ids"], weights=s["weights"])
    tq.exl3_adapter_add(s["x"], s["y"], s["adapters"], s["plan"], out=s["out"])
    return dict(out=s["out"])


# ---------------------------------------------------------------- definition

def _exact_route(s):
    """Row by row on the host, experts as (value, -index) pairs in order."""
    case, E = s["case"], s["case"]["E"]
    rows = s["logits"].double().cpu().tolist()
    bias = s["bias"].double().cpu().tolist() if s["bias"] is not None else [0.0] * E
    size = E // case["groups"]
    all_ids, all_w = [], []
    for l in rows:
        if case["score"] == "softmax":
            top = max(l)
            e = [math.exp(v - top) for v in l]
            tot = math.fsum(e)
            p = [v / tot for v in e]
        else:
            p = [1 / (1 + math.exp(-v)) if v >= 0 else math.exp(v) / (1 + math.exp(v)) for v in l]
        c = [a + b for a, b in zip(p, bias)]
        best = []
        for g in range(case["groups"]):
            top = sorted(c[g * size:(g + 1) * size], reverse=True)
            best.append((-(top[0] if case["group"] == "max" else math.fsum(top[:2])), g))
        left = [e for _, g in sorted(best)[:case["kept"]] for e in range(g * size, (g + 1) * size)]
        ids = sorted(left, key=lambda e: (-c[e], e))[:case["topk"]]
        tot = math.fsum(p[e] for e in ids) if case["renorm"] else 1.0
        all_ids.append(ids)
        all_w.append([p[e] / tot * case["scale"] for e in ids])
    return dict(ids=torch.tensor(all_ids, dtype=torch.int32), weights=torch.tensor(all_w, dtype=torch.float64))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logits":
        y = torch.einsum("tk,ek->te", s["x"].double(), s["w"].double())
        return dict(logits=y if s["bias"] is None else y + s["bias"].double()[None])
    if case["op"] == "route":
        return _exact_route(s)
    # one adapter at a time over all of its rows
    owner = torch.tensor([a for rows, a in s["seqs"] for _ in range(rows)], device="cuda")
    y = s["y"].double()
    for a in range(case["N"]):
        rows = (owner == a).nonzero().flatten()
        if rows.numel():
            h = torch.einsum("tk,rk->tr", s["x"][rows].double(), s["a"][a].double())
            y[rows] += torch.einsum("tr,nr->tn", h * s["scale"][a].double(), s["b"][a].double())
    return dict(out=y)


# ---------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "logits":
        T, k, E = case["T"], case["k"], case["E"]
        return dict(bytes=T * k * 2 + E * k * (4 if case["fp32"] else 2) + T * E * 4 + (E * 4 if case["bias"] else 0),
                    flops=2 * T * k * E)
    if op == "route":
        T, E = case["T"], case["E"]
        return dict(bytes=T * E * (2 if case["fp16"] else 4) + T * case["topk"] * 8 + (E * 4 if case["bias"] else 0),
                    flops=T * E * (4 + case["topk"]))
    seqs, ranks = _sequences(case)
    k, n = case["k"], case["n"]
    T = sum(rows for rows, _ in seqs)
    live = {a for _, a in seqs if a >= 0}
    return dict(bytes=sum(rows for rows, a in seqs if a >= 0) * k * 2 + sum(ranks[a] for a in live) * (k + n) * 2 +
                T * n * 2 * (4 if case["fp32"] else 2) + 8 * len(seqs) + 8 * len(live),
                flops=sum(2 * rows * ranks[a] * (k + n) for rows, a in seqs if a >= 0))
