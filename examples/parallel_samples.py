"""Several samples of each prompt through the attention block of a tensor-parallel
rank group, over the 8-bit cache.

Prompts attend to their own keys and values as the projection gives them, and
write them to the cache; then every prompt is sampled several times.  The samples
share the prompt's whole pages; when they end, pages go back with their last
holder, and now and then the pool is compacted:

    prompt   slot_map, per rank: append, PromptAttention
    sample   pages_fork, per rank: copy
    step     as in decode_block.py, over the 8-bit cache
    finish   pages_release
    compact  pages_compact, per rank: copy

    python examples/parallel_samples.py      # 4 prompts, 8 samples of each; N = 8
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from decode_block import DecodeBlock, rra, serve  # noqa: E402


class SampledBlock(DecodeBlock):
    """A DecodeBlock over 8-bit caches whose requests may share pages."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        pages, size = self.free.numel(), serve.kv8_page_bytes(self.page_tokens, self.hk, self.d)
        self.caches = [serve.KvCache8(torch.empty(pages, size, dtype=torch.uint8, device="cuda"), self.page_tokens, self.hk, self.d)
                       for _ in range(self.ranks)]
        self.prompts = serve.PromptAttention()
        i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.shared, self.moved, self.move_count = i32(pages), i32(pages), i32(1)
        self.move_from, self.move_to = i32(pages), i32(pages)

    def prompt(self, x, new_len, max_len):
        """x [tokens, hidden]: whole prompts of requests that have nothing yet (new_len: 0 for the others)."""
        t = x.shape[0]
        slots, positions = self.slots[:t], self.positions[:t]
        serve.slot_map(self.kv_len, new_len, self.table, self.free, self.free_count, self.page_tokens, kv_len=self.kv_len,
                       cu_new=self.cu, slots=slots, positions=positions, free_left=self.free_count, pages_short=self.short)
        heads = torch.zeros(self.ranks, t, self.hq, self.d, dtype=torch.bfloat16, device="cuda")
        shares = []
        for r in range(self.ranks):
            qkv = (x @ self.wqkv[r]).view(t, self.hq + 2 * self.hk, self.d)
            q, k, v = qkv.split([self.hq, self.hk, self.hk], 1)
            serve.qk_norm_rope(q, k, self.wq, self.wk, self.cos, self.sin, positions, q, k, eps=self.eps)
            self.caches[r].append(k, v, slots)
            self.prompts.attention(q, k, v, heads[r], self.cu[:self.kv_len.numel() + 1], max_len=max_len)
            shares.append(heads[r].view(t, -1) @ self.wo[r])
        outs = [torch.empty_like(x) for _ in range(self.ranks)]
        self.comm.allreduce_residual(shares, [x] * self.ranks, outs)
        return outs[0]

    def sample(self, source, target):
        """Requests `target` (int32) continue requests `source`; both go on from there."""
        copies = torch.empty(2, source.numel(), dtype=torch.int32, device="cuda")
        serve.pages_fork(self.kv_len, source, target, self.table, self.free, self.free_count, self.shared, self.page_tokens,
                         kv_len=self.kv_len, shared_out=self.shared, copy_from=copies[0], copy_to=copies[1],
                         free_left=self.free_count, pages_short=self.short)
        for cache in self.caches:
            cache.copy(copies[0], copies[1])

    def finish(self, new_len):
        """Requests with a negative new_len end; give the same to the next step."""
        serve.pages_release(self.kv_len, new_len, self.table, self.free, self.free_count, self.shared, self.page_tokens,
                            kv_len=self.kv_len, shared_out=self.shared, free_left=self.free_count)

    def compact(self):
        """The pages in use become the pool's first."""
        serve.pages_compact(self.kv_len, self.table, self.free, self.free_count, self.shared, self.page_tokens,
                            table_out=self.table, free_out=self.free, shared_out=self.shared, free_left=self.free_count,
                            moved=self.moved, move_from=self.move_from, move_to=self.move_to, move_count=self.move_count)
        for cache in self.caches:
            cache.copy(self.move_from, self.move_to)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--samples", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--tokens", type=int, default=16)
    a = ap.parse_args()
    rows, n = a.requests * a.samples, a.requests
    most = a.prompt + a.tokens
    block = SampledBlock(a.ranks, a.hidden, q_heads=64, kv_heads=8, max_requests=rows, max_tokens=n * a.prompt,
                         pages=n * (-(-a.prompt // 64)) + rows * (-(-a.tokens // 64) + 2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.randn(n * a.prompt, a.hidden, device="cuda").bfloat16()
    y = block.prompt(x, i32([a.prompt] * n + [0] * (rows - n)), a.prompt)
    # request b's samples: itself, and n + b * (samples - 1) ..
    block.sample(i32([b for b in range(n) for _ in range(a.samples - 1)]), i32(list(range(n, rows))))
    torch.cuda.synchronize()
    print("%d prompts of %d tokens into %d samples: %d pages used" % (n, a.prompt, rows, block.free.numel() - block.free_count.item()))
    x = y.view(n, a.prompt, -1)[:, -1].repeat(a.samples, 1).contiguous()
    new = i32([1] * rows)
    x = block.step(x, new, max_q=1, max_kv=most)
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(a.tokens - 1):
        x = block.step(x, new, max_q=1, max_kv=most)
    torch.cuda.synchronize()
    print("decoding: %.1f us a step" % ((time.perf_counter() - began) / (a.tokens - 1) * 1e6))
    new = i32([1 if b % 2 else -1 for b in range(rows)])
    block.finish(new)
    block.compact()
    block.step(x[new > 0].contiguous(), new, max_q=1, max_kv=most + 1)
    print("half of the samples ended: %d pages used, %d moved, lengths %s" % (
        block.free.numel() - block.free_count.item(), block.move_count.item(), block.kv_len.tolist()))
    assert block.comm.status()[0] == rra.OK and block.short.item() == 0
    assert block.prompts.status() == 0 and all(c.status() == 0 for c in block.caches)
    block.close()


if __name__ == "__main__":
    main()
