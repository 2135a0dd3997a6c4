"""Writes to the 8-bit cache in steps of fixed shape, most of whose slots are padding."""
import numpy as np
import pytest

import more_serve_ref as more
import serve_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def serve():
    from latency_barrier_free_gb300 import serve

    yield serve
    ref.leave_zeros()


def cache_of(serve, num, ps, hk, d):
    return serve.KvCache8(torch.full((num, serve.kv8_page_bytes(ps, hk, d)), 0xA5, dtype=torch.uint8, device="cuda"), ps, hk, d)


# lists of (slots, how often each of them comes one after the other); -1 is padding
LISTS = {
    "padding behind": [(range(3, 9), 1), ([-1], 9000)],
    "padding before": [([-1], 9000), (range(3, 9), 1)],
    "padding inside a run": [(range(3, 6), 1), ([-1], 5000), (range(6, 9), 1), ([10 ** 12], 5000), ([9, 10, 40], 1)],
    "single tokens far apart": [(sum([[64 * i + 5] + [-1] * 1200 for i in range(12)], []), 1)],
    "one slot over and over, with padding": [([21], 300), ([-1], 3000), ([21], 300), ([-1], 70), ([21, 22], 1), ([-1], 4000)],
    "runs that go on behind padding": [([19, 18], 1), ([-1], 2100), ([16, 17], 1), ([-1], 33), ([31, 32], 1), ([-1], 31), ([33], 20)],
    "whole blocks": [(range(0, 640), 1), ([-1], 3000), (range(640, 700), 1), ([-1], 5)],
}


@pytest.mark.parametrize("case", sorted(LISTS))
@pytest.mark.parametrize("hk", [1, 6])
def test_padding(serve, case, hk):
    d, ps, num = 64, 64, 14
    slots = [s for part, n in LISTS[case] for s in list(part) * n]
    rng = np.random.default_rng(len(slots))
    cache = cache_of(serve, num, ps, hk, d)
    pages = cache.pages.cpu().numpy().copy()
    x = torch.from_numpy(rng.standard_normal((len(slots), hk, d)) * 10.0 ** rng.uniform(-2, 2, (len(slots), 1, 1))).cuda().bfloat16()
    if case.startswith("one slot"):  # which of a slot's values stays is not defined: they are the same
        x[:] = x[:1]
    cache.append(x, -x, torch.tensor(slots, device="cuda"))
    cpu = x.double().cpu().numpy()
    more.append8(pages, ps, hk, d, cpu, -cpu, slots)
    assert np.array_equal(cache.pages.cpu().numpy(), pages)


@pytest.mark.parametrize("where", ["behind", "before", "inside a run"])
def test_padding_costs_little(serve, where):
    """131072 slots, three of them real: far from a round trip to memory for each 32 of the others."""
    n = 131072
    slots = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    slots[{"behind": [0, 1, 2], "before": [n - 3, n - 2, n - 1], "inside a run": [0, 1, n - 1]}[where]] = torch.tensor([5, 6, 7], device="cuda")
    cache, x = cache_of(serve, 1, 16, 1, 64), torch.randn(n, 1, 64, device="cuda").bfloat16()
    times = []
    for _ in range(7):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        begin.record()
        cache.append(x, x, slots)
        end.record()
        end.synchronize()
        times.append(begin.elapsed_time(end))
    # 4096 dependent reads of 0.5 us are 2 ms; the CTAs of so many tokens take about 0.1
    assert sorted(times)[3] < 0.7, times
    k, v = torch.empty(3, 1, 64, device="cuda"), torch.empty(3, 1, 64, device="cuda")
    cache.read(torch.tensor([5, 6, 7], device="cuda"), k, v)
    want = x[slots >= 0].float()
    assert ((k - want).abs() <= want.abs() / 16 + 2.0 ** -17 * want.abs().max()).all() and torch.equal(k, v)
