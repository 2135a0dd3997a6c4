"""Scores about as large as they may be, 2^26 in units of log2: rows are finite, and the largest score decides."""
import numpy as np
import pytest

import serve_ref as ref
from test_kv8_gpu import U32, dev, f64, plans, score_error
from test_prompt_gpu import attention

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def serve():
    from latency_barrier_free_gb300 import serve

    yield serve
    ref.leave_zeros()


def scale_of(q, k):
    """Largest scale that is a power of two and leaves scores, times log2(e), below 2^26."""
    most = max(np.abs(q[:, h] @ k[:, h * k.shape[1] // q.shape[1]].T).max() for h in range(q.shape[1]))
    return 2.0 ** np.floor(np.log2(2.0 ** 26 / 1.45 / most))


def check(q, k, v, out, lse, scale):
    _, want_lse, _, dots = attention(q, k, v, scale, True, 0)
    got, group = f64(out), q.shape[1] // k.shape[1]
    tol = score_error(dots, q.shape[2]) + (len(q) + 64) * U32 + 4 * U32 * np.abs(want_lse)
    assert (np.abs(f64(lse) - want_lse) <= tol).all()
    assert np.isfinite(got).all() and (np.abs(got) <= np.maximum.accumulate(np.abs(v), 0).repeat(group, 1) * (1 + 2.0 ** -6)).all()
    # where no other score comes near the largest, its value is the result
    for h in range(q.shape[1]):
        s = np.where(np.tri(len(q), dtype=bool), q[:, h] @ k[:, h // group].T * scale, -np.inf)
        best, order = s.argmax(1), np.sort(s, 1)
        alone = order[:, -1] - order[:, -2] > 2 * tol[:, h] + 40
        assert alone[1:].mean() > 0.5
        want = v[best[alone], h // group]
        # its weight is rounded to the values' type, the sum that it is divided by is not; then the result is rounded: half a step
        # each, of bfloat16 at most (the binary32 product and quotient between them: 2 U32)
        assert (np.abs(got[alone, h] - want) <= (2 * 2.0 ** -8 + 2.0 ** -16 + 2 * U32) * np.abs(want) + 2.0 ** -25).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("max_len", [1, 10 ** 6])  # either kernel
@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (8, 1, 128)])
def test_prompts(serve, hq, hk, d, max_len, dtype):
    rng = np.random.default_rng(1)
    q, k, v = (dev(rng.standard_normal((400, h, d)), dtype) for h in (hq, hk, hk))
    scale = scale_of(f64(q), f64(k))
    prompts, out, lse = serve.PromptAttention(), torch.empty_like(q), torch.empty(400, hq, device="cuda")
    prompts.attention(q, k, v, out, dev(np.array([0, 400], np.int32)), max_len=max_len, scale=scale, lse=lse)
    assert prompts.status() == 0
    check(f64(q), f64(k), f64(v), out, lse, scale)


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (8, 1, 128)])
def test_the_8_bit_cache(serve, hq, hk, d):
    rng = np.random.default_rng(2)
    ps, n = 64, 400
    cache = serve.KvCache8(torch.zeros(7, serve.kv8_page_bytes(ps, hk, d), dtype=torch.uint8, device="cuda"), ps, hk, d)
    k, v = (dev(rng.standard_normal((n, hk, d)).astype(np.float32)) for _ in range(2))
    slots = torch.arange(n, device="cuda")
    cache.append(k, v, slots)
    cache.read(slots, k, v)
    q = dev(rng.standard_normal((n, hq, d)), torch.bfloat16)
    scale = scale_of(f64(q), f64(k))
    for max_q, max_kv in plans(cache, hq, 1).values():
        out, lse = torch.empty_like(q), torch.empty(n, hq, device="cuda")
        cache.attention(q, out, dev(np.array([0, n], np.int32)), dev(np.array([n], np.int32)), torch.arange(7, dtype=torch.int32, device="cuda")[None],
                        max_q=max_q, max_kv=max_kv, scale=scale, lse=lse)
        assert cache.status() == 0
        check(f64(q), f64(k), f64(v), out, lse, scale)
