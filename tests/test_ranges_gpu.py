"""Query ranges at the ends of 32 bits, by every attention kernel of either cache: clamped, nothing outside the buffers is read
or written."""
import numpy as np
import pytest

import serve_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def serve():
    from latency_barrier_free_gb300 import serve

    yield serve
    ref.leave_zeros()


@pytest.mark.parametrize("kind", ["KvCache", "KvCache8"])
def test_the_smallest_and_largest_range_ends(serve, kind):
    d, ps, hk, hq, t = 64, 16, 2, 4, 40
    size = serve.kv_page_bytes(ps, hk, d) if kind == "KvCache" else serve.kv8_page_bytes(ps, hk, d)
    cache = getattr(serve, kind)(torch.zeros(8, size, dtype=torch.uint8, device="cuda"), ps, hk, d)
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(t, hk, d, generator=gen, device="cuda") for _ in range(2))
    cache.append(k, v, torch.arange(t, device="cuda"))
    q = torch.randn(t, hq, d, generator=gen, device="cuda").bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table, kv = i32([[0, 1, 2]] * 2), i32([t, t])
    low, high = -2 ** 31, 2 ** 31 - 1
    for max_q, max_kv in ((1, 64), (1, 10 ** 5), (4, 10 ** 9), (32, 64), (10 ** 6, 10 ** 9)):
        want = torch.full_like(q, 7.0)
        cache.attention(q, want, i32([0, t, t]), kv, table, max_q=max_q, max_kv=max_kv)
        for cu in ([low, high, high], [-1, t, low], [high, low, 0], [t, low, low], [3, low, high]):
            out = torch.full((t + 8, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
            cache.attention(q, out[4:-4], i32(cu), kv, table, max_q=max_q, max_kv=max_kv)
            torch.cuda.synchronize()
            assert (out[:4] == 7).all() and (out[-4:] == 7).all()
            if cu[0] <= 0:
                assert torch.equal(out[4:-4], want)
    assert cache.status() == 0
