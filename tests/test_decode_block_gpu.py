"""The operators together, as the decode-step example runs them, against plain
attention in 64 bits over what the ranks' caches hold."""
import os
import sys

import numpy as np
import pytest

import serve_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

U8 = 2.0 ** -8


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import decode_block

    yield decode_block
    ref.leave_zeros()


def f64(t):
    return t.detach().cpu().double().numpy()


def plain_step(block, x, kv, new):
    """The block on x with the lengths `kv` after the step; bfloat16 where the step rounds, 64 bits elsewhere."""
    x = f64(x)
    rnd = lambda a: f64(torch.from_numpy(a).bfloat16())  # noqa: E731
    total = np.zeros_like(x)
    at = 0
    positions, tokens = [], []
    for b, n in enumerate(new):
        n = max(int(n), 0)
        positions += range(kv[b] - n, kv[b])
        tokens.append((at, n))
        at += n
    table = block.table.cpu().numpy()
    for r in range(block.ranks):
        qkv = rnd(x @ f64(block.wqkv[r])).reshape(len(x), -1, block.d)
        q, _ = ref.norm_rope(qkv[:, :block.hq], f64(block.wq), f64(block.cos), f64(block.sin), np.array(positions), block.eps, False)
        q, o = rnd(q), np.zeros((len(x), block.hq, block.d))
        pages = block.caches[r].pages.cpu().numpy()
        for b, (at, n) in enumerate(tokens):
            if n == 0:
                continue
            i = np.arange(kv[b])
            slots = table[b, i // block.page_tokens].astype(np.int64) * block.page_tokens + i % block.page_tokens
            k, v = ref.read_pages(pages, block.page_tokens, block.hk, block.d, slots)
            o[at:at + n], *_ = ref.attention(q[at:at + n], k, v, int(kv[b]), block.d ** -0.5, True, 0)
        total += rnd(rnd(o).reshape(len(x), -1) @ f64(block.wo[r]))
    return total + x


def test_prompts_then_tokens(example):
    block = example.DecodeBlock(ranks=2, hidden=256, q_heads=8, kv_heads=2, head_dim=64, pages=24, page_tokens=16, max_requests=4,
                                max_pages=10, max_tokens=256, max_position=512)
    try:
        gen = torch.Generator(device="cuda").manual_seed(1)
        kv = np.zeros(4, np.int64)
        # prompts, tokens, one request ends, another takes its place, a step with a request that has nothing
        for new in ([70, 33, 1, 16], [1, 1, 1, 1], [1, -1, 1, 1], [1, 40, 1, 1], [1, 1, 0, 1]):
            t = sum(max(n, 0) for n in new)
            x = torch.randn(t, 256, generator=gen, device="cuda").bfloat16()
            y = block.step(x, torch.tensor(new, dtype=torch.int32, device="cuda"), max_q=max(new), max_kv=128)
            torch.cuda.synchronize()
            kv = np.array([0 if n < 0 else k + n for k, n in zip(kv, new)])
            assert block.kv_len.tolist() == kv.tolist() and block.short.item() == 0
            want = plain_step(block, x, kv, new)
            # the block's own share is of size about 1; every product's result is rounded to bfloat16, and so are the
            # products' inputs that differ by a rounding here and there: a few roundings of values of that size
            assert np.abs(f64(y) - want).max() <= 8 * U8 * max(1.0, np.abs(want).max()), np.abs(f64(y) - want).max()
        held = sum(-(-int(k) // 16) for k in kv)
        assert block.free_count.item() == 24 - held
        assert block.comm.status()[0] == 0 and all(c.status() == 0 for c in block.caches)
    finally:
        block.close()


def test_a_decode_step_from_a_graph(example):
    """Replays advance lengths, pages and slots on the GPU; the result is that of the same steps enqueued one by one."""
    def run(graph):
        block = example.DecodeBlock(ranks=2, hidden=256, q_heads=4, kv_heads=2, head_dim=128, pages=24, page_tokens=16,
                                    max_requests=2, max_pages=8, max_tokens=64, max_position=512)
        x = torch.randn(20, 256, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
        y = block.step(x, torch.tensor([13, 7], dtype=torch.int32, device="cuda"), max_q=13, max_kv=64)
        x = y[[12, 19]].contiguous()
        new = torch.ones(2, dtype=torch.int32, device="cuda")
        x.copy_(block.step(x, new, max_q=1, max_kv=64))
        if graph:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                x.copy_(block.step(x, new, max_q=1, max_kv=64))
            for _ in range(20):
                g.replay()
        else:
            for _ in range(20):
                x.copy_(block.step(x, new, max_q=1, max_kv=64))
        torch.cuda.synchronize()
        state = x.clone(), block.kv_len.tolist(), block.free_count.item(), block.short.item()
        block.close()
        return state

    a, b = run(False), run(True)
    assert a[1:] == b[1:] == ([34, 28], 24 - 5, 0)
    assert torch.equal(a[0], b[0])


def test_padding_of_a_step_stays_as_it_was(example):
    """A step of fixed shape with fewer new tokens than rows, over memory that held NaN."""
    block = example.DecodeBlock(ranks=2, hidden=256, q_heads=8, kv_heads=2, head_dim=64, pages=24, page_tokens=16, max_requests=4,
                                max_pages=10, max_tokens=64, max_position=512)
    try:
        gen = torch.Generator(device="cuda").manual_seed(5)
        x = torch.randn(40, 256, generator=gen, device="cuda").bfloat16()
        kv = np.zeros(4, np.int64)
        for new in ([9, 0, 20, 1], [1, 1, -1, 0]):
            nan = [torch.full((n,), float("nan"), dtype=torch.bfloat16, device="cuda") for n in (40 * 4 * 64, 40 * 256) for _ in range(8)]
            del nan
            y = block.step(x, torch.tensor(new, dtype=torch.int32, device="cuda"), max_q=max(new), max_kv=64)
            torch.cuda.synchronize()
            kv = np.array([0 if n < 0 else k + n for k, n in zip(kv, new)])
            t = sum(max(n, 0) for n in new)
            assert torch.equal(y[t:], x[t:])
            want = plain_step(block, x[:t], kv, new)
            assert np.abs(f64(y[:t]) - want).max() <= 8 * U8 * max(1.0, np.abs(want).max())
    finally:
        block.close()
