"""Prompts, their samples, decode steps, ends and compaction together, as the example runs them, against plain attention in 64
bits over what the ranks' caches hold."""
import os
import subprocess
import sys

import numpy as np
import pytest

import more_serve_ref as more
import serve_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

U8 = 2.0 ** -8


@pytest.fixture(scope="module")
def example():
    import __graft_entry__

    __graft_entry__.build()
    import parallel_samples

    yield parallel_samples
    ref.leave_zeros()


def f64(t):
    return t.detach().cpu().double().numpy()


def held(block, r, b, kv):
    """Keys and values of request b on rank r."""
    i = np.arange(int(kv[b]))
    table = block.table.cpu().numpy()
    slots = table[b, i // block.page_tokens].astype(np.int64) * block.page_tokens + i % block.page_tokens
    return more.read8(block.caches[r].pages.cpu().numpy(), block.page_tokens, block.hk, block.d, slots)


def plain_step(block, x, kv, new, own=False):
    """The block on x with the lengths `kv` after the step; with `own` prompts see their keys and values before the cache."""
    x = f64(x)
    rnd = lambda a: f64(torch.from_numpy(a).bfloat16())  # noqa: E731
    total, at, positions, tokens = np.zeros_like(x), 0, [], []
    for b, n in enumerate(new):
        n = max(int(n), 0)
        positions += range(kv[b] - n, kv[b])
        tokens.append((at, n))
        at += n
    for r in range(block.ranks):
        qkv = rnd(x @ f64(block.wqkv[r])).reshape(len(x), -1, block.d)
        norm = lambda y, w: rnd(ref.norm_rope(y, f64(w), f64(block.cos), f64(block.sin), np.array(positions), block.eps, False)[0])  # noqa: E731
        q, keys, values = norm(qkv[:, :block.hq], block.wq), norm(qkv[:, block.hq:-block.hk], block.wk), qkv[:, -block.hk:]
        o = np.zeros((len(x), block.hq, block.d))
        for b, (at, n) in enumerate(tokens):
            if n:
                k, v = (keys[at:at + n], values[at:at + n]) if own else held(block, r, b, kv)
                o[at:at + n], *_ = ref.attention(q[at:at + n], k, v, int(kv[b]), block.d ** -0.5, True, 0)
        total += rnd(rnd(o).reshape(len(x), -1) @ f64(block.wo[r]))
    return total + x


def test_prompts_samples_ends_and_compaction(example):
    block = example.SampledBlock(ranks=2, hidden=256, q_heads=8, kv_heads=2, head_dim=64, pages=40, page_tokens=16, max_requests=6,
                                 max_pages=10, max_tokens=256, max_position=512)
    try:
        gen = torch.Generator(device="cuda").manual_seed(1)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        fresh = lambda t: torch.randn(t, 256, generator=gen, device="cuda").bfloat16()  # noqa: E731
        kv = np.zeros(6, np.int64)

        def check(x, y, new, own=False):
            torch.cuda.synchronize()
            assert block.kv_len.tolist() == kv.tolist() and block.short.item() == 0
            want = plain_step(block, x, kv, new, own)
            # products' results and inputs are rounded to bfloat16: a few roundings of values of that size
            assert np.abs(f64(y) - want).max() <= 8 * U8 * max(1.0, np.abs(want).max())

        def used():
            return 40 - block.free_count.item()

        new = [70, 33, 0, 0, 0, 0]
        x, kv = fresh(103), np.array(new)
        check(x, block.prompt(x, i32(new), 70), new, own=True)
        assert used() == 8
        block.sample(i32([0, 0, 1, 0]), i32([2, 3, 4, 5]))
        kv[[2, 3, 5]], kv[4] = 70, 33
        torch.cuda.synchronize()
        assert used() == 12 and block.shared.sum().item() == 3 * 4 + 2
        for r in range(2):
            for a, b in ((0, 2), (0, 3), (1, 4), (0, 5)):
                assert np.array_equal(held(block, r, a, kv), held(block, r, b, kv))
        for _ in range(3):  # each goes its own way
            x, new = fresh(6), [1] * 6
            kv = kv + 1
            check(x, block.step(x, i32(new), max_q=1, max_kv=128), new)
        before = [[held(block, r, b, kv) for b in range(6)] for r in range(2)]
        assert not np.array_equal(before[0][0], before[0][2])
        new = [-1, 1, 1, -1, -1, 1]
        block.finish(i32(new))
        kv[[0, 3, 4]] = 0
        block.compact()
        torch.cuda.synchronize()
        # 0, 3 and 4 have ended: the whole pages of 0 stay with 2 and 5, those of 4 with 1
        assert block.kv_len.tolist() == kv.tolist() and used() == 4 + 2 + 3 and block.shared.sum().item() == 4
        assert block.free.tolist()[:31] == list(range(39, 8, -1))
        for r in range(2):
            for b in (1, 2, 5):
                assert np.array_equal(held(block, r, b, kv), before[r][b])
        x, kv = fresh(3), kv + np.array([0, 1, 1, 0, 0, 1])
        check(x, block.step(x, i32(new), max_q=1, max_kv=128), new)
        # the rows that ended take prompts again
        new = [20, 0, 0, 90, 0, 0]
        x, kv = fresh(110), kv + np.array(new)
        check(x, block.prompt(x, i32(new), 90), new, own=True)
        block.finish(i32([-1] * 6))
        torch.cuda.synchronize()
        assert used() == 0 and block.shared.abs().sum().item() == 0 and sorted(block.free.tolist()) == list(range(40))
        assert block.prompts.status() == 0 and all(c.status() == 0 for c in block.caches) and block.comm.status()[0] == 0
    finally:
        block.close()


def test_the_example_runs():
    p = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "parallel_samples.py"), "--prompt", "200", "--hidden", "512"],
                       capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    assert "4 prompts of 200 tokens into 32 samples" in p.stdout
