"""The attention block of a tensor-parallel decode step, over N virtual ranks.

Every rank holds its share of the heads, of the projections and of the 4-bit
key/value cache; one page table serves all ranks.  A step of the serving loop is

    slot_map                                         once
    per rank:  x Wqkv, qk_norm_rope, append, attention, o Wo
    AllReduce of the ranks' shares + residual        once

and holds for prompts (many new tokens of a request) and for single tokens alike.
The step of a batch that only decodes is replayed from a CUDA graph: lengths,
pages and slots change on the GPU, not on the host.

    python examples/decode_block.py          # a prompt, then 32 tokens; N = 8
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from latency_barrier_free_gb300 import rra, serve  # noqa: E402


class DecodeBlock:
    """One attention block on `ranks` virtual ranks of the current GPU."""

    def __init__(self, ranks, hidden, q_heads, kv_heads, head_dim=128, pages=256, page_tokens=64, max_requests=64,
                 max_pages=64, max_tokens=4096, max_position=65536, theta=500000.0, eps=1e-6, seed=0):
        assert q_heads % ranks == 0 and kv_heads % ranks == 0
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.ranks, self.hq, self.hk, self.d = ranks, q_heads // ranks, kv_heads // ranks, head_dim
        self.hidden, self.page_tokens, self.eps = hidden, page_tokens, eps
        rows = (self.hq + 2 * self.hk) * head_dim
        self.wqkv = [(rand(hidden, rows) / hidden ** 0.5).bfloat16() for _ in range(ranks)]
        self.wo = [(rand(self.hq * head_dim, hidden) / (q_heads * head_dim) ** 0.5).bfloat16() for _ in range(ranks)]
        self.wq, self.wk = ((1 + 0.1 * rand(head_dim)).bfloat16() for _ in range(2))
        angle = torch.arange(max_position, dtype=torch.float64)[:, None] \
            * theta ** (-torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim)
        self.cos, self.sin = angle.cos().float().cuda(), angle.sin().float().cuda()
        size = serve.kv_page_bytes(page_tokens, self.hk, head_dim)
        self.caches = [serve.KvCache(torch.empty(pages, size, dtype=torch.uint8, device="cuda"), page_tokens, self.hk, head_dim)
                       for _ in range(ranks)]
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        # the requests' state: lengths, pages, and the stack of free pages
        self.kv_len, self.table = i32(max_requests), i32(max_requests, max_pages)
        self.free = torch.arange(pages, dtype=torch.int32, device="cuda")
        self.free_count, self.short = torch.full((1,), pages, dtype=torch.int32, device="cuda"), i32(1)
        self.new_len, self.cu = i32(max_requests), i32(max_requests + 1)
        self.slots, self.positions = torch.zeros(max_tokens, dtype=torch.int64, device="cuda"), i32(max_tokens)
        self.comm = rra.Comm(ranks, max_tokens * hidden * 2)

    def step(self, x, new_len, max_q, max_kv):
        """x [tokens, hidden]: the new tokens of every request, in the order of the
        requests, and padding after them, if any; new_len [requests] int32 on the GPU
        (negative: the request ends).  Returns x plus the block's output; padding as
        it was."""
        t, n = x.shape[0], self.kv_len.numel()
        slots, positions = self.slots[:t], self.positions[:t]
        serve.slot_map(self.kv_len, new_len, self.table, self.free, self.free_count, self.page_tokens, kv_len=self.kv_len,
                       cu_new=self.cu, slots=slots, positions=positions, free_left=self.free_count, pages_short=self.short)
        # zeros: the attention leaves the rows of padding as they are
        heads = torch.zeros(self.ranks, t, self.hq, self.d, dtype=torch.bfloat16, device="cuda")
        shares = []
        for r in range(self.ranks):
            qkv = (x @ self.wqkv[r]).view(t, self.hq + 2 * self.hk, self.d)
            q, k, v = qkv.split([self.hq, self.hk, self.hk], 1)
            serve.qk_norm_rope(q, k, self.wq, self.wk, self.cos, self.sin, positions, q, k, eps=self.eps)
            self.caches[r].append(k, v, slots)
            self.caches[r].attention(q, heads[r], self.cu[:n + 1], self.kv_len, self.table, max_q=max_q, max_kv=max_kv)
            shares.append(heads[r].view(t, -1) @ self.wo[r])
        outs = [torch.empty_like(x) for _ in range(self.ranks)]
        self.comm.allreduce_residual(shares, [x] * self.ranks, outs)
        return outs[0]

    def close(self):
        self.comm.close()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--tokens", type=int, default=32)
    a = ap.parse_args()
    block = DecodeBlock(a.ranks, a.hidden, q_heads=64, kv_heads=8, max_requests=a.requests,
                        max_tokens=a.requests * a.prompt, pages=a.requests * (-(-(a.prompt + a.tokens) // 64) + 1))
    new = torch.full((a.requests,), a.prompt, dtype=torch.int32, device="cuda")
    x = torch.randn(a.requests * a.prompt, a.hidden, device="cuda").bfloat16()
    most = a.prompt + a.tokens
    y = block.step(x, new, max_q=a.prompt, max_kv=a.prompt)
    torch.cuda.synchronize()
    print("prompts: %d requests of %d tokens, |y| %.3f" % (a.requests, a.prompt, y.float().norm() / y.numel() ** 0.5))

    new.fill_(1)
    x = y.view(a.requests, a.prompt, -1)[:, -1].contiguous()
    for _ in range(3):  # lengths, pages and slots advance with every call, captured or not
        x.copy_(block.step(x, new, max_q=1, max_kv=most))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        x.copy_(block.step(x, new, max_q=1, max_kv=most))
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(a.tokens - 3):
        graph.replay()
    torch.cuda.synchronize()
    print("decoding: %d tokens of %d requests, %.1f us a step (%d ranks on one GPU), lengths %s, %d pages left" % (
        a.tokens - 3, a.requests, (time.perf_counter() - began) / (a.tokens - 3) * 1e6, a.ranks, block.kv_len.tolist(),
        block.free_count.item()))
    assert block.comm.status()[0] == rra.OK and all(c.status() == 0 for c in block.caches) and block.short.item() == 0
    block.close()


if __name__ == "__main__":
    main()
