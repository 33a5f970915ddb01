"""The attention half of a decoder layer on EXL3 weights: a prompt in chunks,
then decode steps from a CUDA graph.

    x -> q, k, v linears (fused shards) -> head norms, rotary positions and the
    append to a paged cache (one launch) -> attention over the cache -> output
    linear

Run:  python examples/attention_block.py            (hidden 5120, 40/8 heads of 128)
      python examples/attention_block.py --small    (hidden 512, 4/2 heads of 128)

The weights are random; the run prints the time of a chunk and of a step and
how far the last step is from the same layer done with plain torch operations
on the dequantised path's projections.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import trellis_quantized_gb300 as tq  # noqa: E402


class AttentionBlock:
    """q, k, v and output linears of K-bit trellis weights around paged attention."""

    def __init__(self, hidden, heads_q, heads_kv, head_dim, K=4, pages=64, page_size=64, max_pages=32, batch=1,
                 base=1e6, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.hidden, self.Hq, self.Hkv, self.D, self.K = hidden, heads_q, heads_kv, head_dim, K
        self.widths = (heads_q * head_dim, heads_kv * head_dim, heads_kv * head_dim)

        def words(k, n):
            return torch.randint(-2 ** 15, 2 ** 15, (k // 16, n // 16, 16 * K), dtype=torch.int16, device="cuda",
                                 generator=g)

        def signs(n):
            return (torch.randint(0, 2, (n,), device="cuda", generator=g) * 2 - 1).half()

        self.qkv = torch.cat([words(hidden, n).reshape(-1) for n in self.widths])
        self.qkv_suh = torch.stack([signs(hidden) for _ in self.widths])
        # the trellis values have a standard deviation near one: scale the outputs back to that of x
        self.qkv_svh = torch.cat([signs(n) for n in self.widths]) * hidden ** -0.5
        self.o = words(heads_q * head_dim, hidden)
        self.o_suh, self.o_svh = signs(heads_q * head_dim), signs(hidden) * (heads_q * head_dim) ** -0.5
        norm = lambda: (1 + 0.1 * torch.randn(head_dim, generator=g, device="cuda")).half()
        freq, mag = tq.exl3_rope_frequencies(head_dim, base)
        self.q_norm, self.k_norm, self.inv_freq = norm(), norm(), freq.cuda()
        self.transform = tq.head_transform(self.q_norm, self.k_norm, 1e-6, self.inv_freq, magnitude=mag)
        shape = (pages, page_size, heads_kv, head_dim)
        self.k, self.v = (torch.zeros(shape, dtype=torch.float16, device="cuda") for _ in range(2))
        self.cache = tq.kv_cache(self.k, self.v)
        assert batch * max_pages <= pages
        self.table = torch.arange(batch * max_pages, dtype=torch.int32, device="cuda").view(batch, max_pages)
        # one workspace for every call of the layer, kept as long as graphs that use it
        rows = 4096
        need = [tq.exl3_linear_shards_var_workspace_size(m, hidden, self.widths, K) for m in (1, 128, rows)]
        need += [tq.exl3_linear_workspace_size(m, heads_q * head_dim, hidden, K) for m in (1, 128, rows)]
        need += [tq.exl3_paged_attention_workspace_size(m, heads_q, heads_kv, head_dim, batch) for m in (1, batch, rows)]
        self.ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")
        tq.exl3_workspace_clear(self.ws)

    def project(self, x):
        """q, k and v of x [T, hidden] as [T, heads, D] views of the shards' output."""
        T = x.shape[0]
        y = tq.exl3_linear_shards_var(x, self.qkv, self.qkv_suh, self.qkv_svh, self.widths, self.K,
                                      workspace_buf=self.ws)
        parts = torch.split(y, [T * n for n in self.widths])
        return [p.view(T, n // self.D, self.D) for p, n in zip(parts, self.widths)]

    def __call__(self, x, batch):
        q, k, v = self.project(x)
        tq.exl3_qkv_append(q, k, v, batch, self.cache, self.transform, q_out=q, workspace_buf=self.ws)
        a = tq.exl3_paged_attention(q, batch, self.cache, workspace_buf=self.ws)
        return tq.exl3_linear(a.view(x.shape[0], -1), self.o, self.o_suh, self.o_svh, self.K, workspace_buf=self.ws)


def plain_attention(block, x_all, chunks):
    """The attention of the last token in fp64, from the projections of every token."""
    q, k, v = (torch.cat(p) for p in zip(*[block.project(x_all[s:e]) for s, e in chunks]))
    pos = torch.arange(x_all.shape[0], device="cuda").double()

    def rotate(t, w):
        t = t.double()
        t = t / torch.sqrt(t.square().mean(-1, keepdim=True) + 1e-6) * w.double()
        ang = pos[:, None, None] * block.inv_freq.double()
        a, b = t.chunk(2, -1)
        return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)

    q, k, v = rotate(q, block.q_norm)[-1], rotate(k, block.k_norm), v.double()
    G = block.Hq // block.Hkv
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    p = torch.softmax(torch.einsum("hd,jhd->hj", q, k) * block.D ** -0.5, -1)
    return torch.einsum("hj,jhd->hd", p, v)


def run(hidden, heads_q, heads_kv, head_dim, prompt, chunk, steps):
    """Prompt in chunks, then `steps` graph replays; returns (relative error, ms per chunk, us per step)."""
    block = AttentionBlock(hidden, heads_q, heads_kv, head_dim, pages=64, max_pages=64)
    assert prompt + steps + 1 <= 64 * 64
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x_all = torch.randn((prompt + steps, hidden), generator=g, device="cuda").half()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    chunks = [(s, min(prompt, s + chunk)) for s in range(0, prompt, chunk)]
    ev[0].record()
    for s, e in chunks:
        block(x_all[s:e], tq.paged_batch(i32([0, e - s]), i32([e]), block.table))
    ev[1].record()
    # one captured step serves every length: the kernels read kv_len on the device
    q_start, kv_len = i32([0, 1]), i32([prompt + 1])
    x = x_all[prompt:prompt + 1].clone()
    batch = tq.paged_batch(q_start, kv_len, block.table)
    block(x, batch)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(x, batch)
    ev[2].record()
    for i in range(steps):
        x.copy_(x_all[prompt + i:prompt + i + 1])
        kv_len.fill_(prompt + i + 1)
        graph.replay()
    ev[3].record()
    torch.cuda.synchronize()
    err = tq.exl3_check_device_error(block.ws)
    assert err == 0, f"device error word {err}"
    # the same layer on plain attention
    want = plain_attention(block, x_all, chunks + [(i, i + 1) for i in range(prompt, prompt + steps)])
    want = tq.exl3_linear(want.half().view(1, -1), block.o, block.o_suh, block.o_svh, block.K)
    rel = float((y.double() - want.double()).norm() / want.double().norm())
    return rel, ev[0].elapsed_time(ev[1]) / len(chunks), ev[2].elapsed_time(ev[3]) * 1e3 / steps


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--small", action="store_true")
    small = ap.parse_args().small
    shape = dict(hidden=512, heads_q=4, heads_kv=2, head_dim=128, prompt=300, chunk=128, steps=5) if small else \
        dict(hidden=5120, heads_q=40, heads_kv=8, head_dim=128, prompt=4000, chunk=2000, steps=50)
    rel, ms, us = run(**shape)
    print(f"{shape}\nchunk {ms:.3f} ms, step {us:.1f} us, last step against plain attention: rel-L2 {rel:.2e}")
