"""The 8-bit cache and the attention over it on a GPU, against their definitions in 64 bits."""
import numpy as np
import pytest

import more_serve_ref as more
import serve_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# half steps: off by at most these relative to the value
U32, U16, U8 = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8


@pytest.fixture(scope="module")
def serve():
    from latency_barrier_free_gb300 import serve

    yield serve
    ref.leave_zeros()


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.double().cpu().numpy()


def cache_of(serve, num, ps, hk, d, fill=0xA5):
    return serve.KvCache8(torch.full((num, serve.kv8_page_bytes(ps, hk, d)), fill, dtype=torch.uint8, device="cuda"), ps, hk, d)


# ------------------------------------------------------- write and read --
STORES = {
    # name: d, ps, hk, dtype, slots of each call
    "one token": (64, 16, 1, "fp32", [[17]]),
    "a block": (128, 16, 2, "bf16", [list(range(16, 32))]),
    "a block in any order": (64, 32, 1, "bf16", [[5, 3, 0, 1, 2, 4, 15, 7]]),
    "a block by and by": (128, 64, 3, "fp32", [[64], [65, 66], [67, 68, 69, 70, 71, 72], [73], list(range(74, 85))]),
    "runs over several blocks": (64, 64, 5, "bf16", [list(range(7, 60)) + list(range(130, 131)) + list(range(64, 100))]),
    "slots outside": (128, 16, 4, "bf16", [[-1, 3, -7, 10 ** 6, 48, 49, -1, 2 ** 40, 50]]),
    "begun anew": (64, 16, 2, "fp32", [list(range(16)), [0], [1, 2]]),
    "many tokens": (128, 48, 8, "bf16", [list(range(0, 700)), list(range(700, 960))]),
    "heads that are not multiples of four": (64, 16, 7, "fp32", [list(range(0, 400)), [400], [401, 402]]),
}


@pytest.mark.parametrize("case", sorted(STORES))
def test_append_and_read(serve, case):
    d, ps, hk, dtype, calls = STORES[case]
    rng = np.random.default_rng(5)
    num = -(-1000 // ps)
    cache = cache_of(serve, num, ps, hk, d)
    pages = cache.pages.cpu().numpy().copy()
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    for i, slots in enumerate(calls):
        wide = rng.standard_normal((len(slots), hk + 1, 2 * d)) * 10.0 ** rng.uniform(-3, 3, (len(slots), 1, 1))
        x = dev(wide, dt)
        k, v = x[:, :hk, :d], x[:, 1:, d:]  # strided
        cache.append(k, v, dev(np.array(slots, np.int64)))
        more.append8(pages, ps, hk, d, f64(k), f64(v), slots)
        torch.cuda.synchronize()
        got = cache.pages.cpu().numpy()
        assert np.array_equal(got, pages), (case, i, np.argwhere(got != pages)[:5])
    slots = [s for c in calls for s in c] + [-1, num * ps]
    want = more.read8(pages, ps, hk, d, slots)
    k, v = (torch.full((len(slots), hk, d), 7.0, device="cuda") for _ in range(2))
    cache.read(dev(np.array(slots, np.int64)), k, v)
    assert np.array_equal(f64(k), want[0]) and np.array_equal(f64(v), want[1])
    kb, vb = (torch.full((len(slots), hk, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache.read(dev(np.array(slots, np.int64)), kb, vb)
    assert torch.equal(kb, k.bfloat16()) and torch.equal(vb, v.bfloat16())


@pytest.mark.parametrize("tokens", [500, 700, 1300, 2500, 5000])
def test_runs_that_end_anywhere_among_a_ctas_tokens(serve, tokens):
    """Runs of 1 to 40 neighbours from anywhere in a page, with skipped slots between: a CTA takes more tokens the more there are."""
    d, ps, hk, num = 64, 64, 1, 3000
    rng = np.random.default_rng(tokens)
    slots, pages_left = [], rng.permutation(num).tolist()
    while len(slots) < tokens:
        first = int(rng.integers(0, ps))
        run = (pages_left.pop() * ps + np.arange(first, min(ps, first + int(rng.integers(1, 41))))).tolist()
        if rng.integers(0, 4) == 0:
            run.insert(int(rng.integers(0, len(run) + 1)), -1)
        slots += run
    slots = slots[:tokens]
    cache = cache_of(serve, num, ps, hk, d)
    pages = cache.pages.cpu().numpy().copy()
    x = dev(rng.standard_normal((tokens, hk, 2 * d)) * 10.0 ** rng.uniform(-3, 3, (tokens, 1, 1)), torch.bfloat16)
    cache.append(x[..., :d], x[..., d:], dev(np.array(slots, np.int64)))
    more.append8(pages, ps, hk, d, f64(x[..., :d]), f64(x[..., d:]), slots)
    assert np.array_equal(cache.pages.cpu().numpy(), pages)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_what_rounding_does(serve, dtype):
    """Ties, the largest and smallest exponents, infinities, NaN, zeros of both signs."""
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    d, ps, hk = 64, 16, 1
    rows = [
        [448.0, 1.0625, 1.1875, -1.0625, 2.0 ** -10, 3 * 2.0 ** -10, -0.0, 0.0],  # ties in unit 1
        [np.nan, np.inf, -np.inf, 1.0, 2.0, 3.0, -448.0, 0.0],
        [3e38, -3e38, 1e30, 1.0, np.nan, 0.0, 2.0 ** 41, 2.0 ** 40],
        [1e-30, -1e-20, 2.0 ** -41, 2.0 ** -42, 1.5 * 2.0 ** -41, 0.0, 0.0, 0.0],
        [np.inf] * 8,
        [0.0] * 8,
        [449.0 if dtype == "fp32" else 450.0, 1.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0],
    ]
    cache = cache_of(serve, len(rows), ps, hk, d, 0)
    pages = cache.pages.cpu().numpy().copy()
    x = dev(np.tile(np.array(rows), (1, d // 8))[:, None, :], dt)
    slots = [16 * i for i in range(len(rows))]
    cache.append(x, -x, dev(np.array(slots, np.int64)))
    more.append8(pages, ps, hk, d, f64(x), f64(-x), slots)
    assert np.array_equal(cache.pages.cpu().numpy(), pages)
    # later tokens of other sizes: the codes that are there are rounded again
    for by in (2.0 ** -9, 3.0, 2.0 ** 20):
        y = (x * by).to(dt)
        slots = [s + 1 for s in slots]
        cache.append(y, y, dev(np.array(slots, np.int64)))
        more.append8(pages, ps, hk, d, f64(y), f64(y), slots)
        assert np.array_equal(cache.pages.cpu().numpy(), pages), by


def test_a_value_is_within_its_bound(serve):
    """2^-4 of itself, or 2^-10 units for the write and each raise of the exponent."""
    d, ps, hk = 128, 16, 2
    rng = np.random.default_rng(2)
    cache = cache_of(serve, 1, ps, hk, d)
    x = (rng.standard_normal((16, hk, d)) * 2.0 ** np.arange(16)[:, None, None]).astype(np.float32)  # each raises it
    for i in range(16):
        cache.append(dev(x[i:i + 1]), dev(x[i:i + 1]), dev(np.array([i], np.int64)))
    k, v = torch.empty(16, hk, d, device="cuda"), torch.empty(16, hk, d, device="cuda")
    cache.read(dev(np.arange(16)), k, v)
    unit = np.abs(x).max((0, 2), keepdims=True) / 224  # 2^e is at most this
    for got in (f64(k), f64(v)):
        assert (np.abs(got - x) <= 2.0 ** -4 * np.abs(x) + (2.0 ** -10 + 15 * 2.0 ** -10) * unit).all()


def test_slots_that_occur_twice_get_either_tokens_values(serve):
    d, ps, hk = 64, 16, 3
    cache = cache_of(serve, 4, ps, hk, d)
    t = 100
    x = dev(np.repeat(2.0 ** (np.arange(t) % 8), hk * d).reshape(t, hk, d).astype(np.float32))
    cache.append(x, x, dev(np.full(t, 18, np.int64)))
    k, v = torch.empty(1, hk, d, device="cuda"), torch.empty(1, hk, d, device="cuda")
    cache.read(dev(np.array([18], np.int64)), k, v)
    allowed = torch.tensor([2.0 ** i for i in range(8)], device="cuda")
    assert torch.isin(k, allowed).all() and torch.isin(v, allowed).all()


# ------------------------------------------------------------- attention --
def score_error(dots, d):
    """A score is a sum of d products in binary32, scaled three times; times log2(e), rounded, and exponentiated
    (2^-22 relative): an absolute error in the exponent."""
    return (d + 8) * 2 * U32 * dots + 2.0 ** -21


def check_out(got, want, mean, dots, d, kv, largest):
    # A weight is rounded to binary16: by half a step, or by 2^-25 where the largest is at least 2^7 / 2 (448 units of a block
    # are at most twice its largest value: kv * 2^-25 / 2^6 * 2); sums of kv terms in binary32.
    e = (U16 + 2 * score_error(dots, d) + (kv + 64) * U32)[..., None]
    tol = U8 * np.abs(want) + (1 + U8) * (e * mean + kv * 2.0 ** -30 * largest) + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (bad.sum(), np.max(np.abs(got - want)[bad] / tol[bad]))


CASES = {
    # name: hq, hk, d, ps, query counts, key counts, causal, window
    "one token, one key": (1, 1, 64, 16, [1], [1], True, 0),
    "one token": (8, 1, 128, 64, [1], [77], True, 0),
    "groups of 7, ragged": (14, 2, 64, 16, [1, 1, 1, 1], [1, 15, 16, 333], True, 0),
    "nothing to see": (8, 2, 128, 32, [1, 1, 1], [0, 40, 0], True, 0),
    "no queries": (4, 2, 64, 16, [0, 2, 0], [9, 20, 0], True, 0),
    "more queries than keys": (4, 4, 128, 16, [9, 3], [4, 3], True, 0),
    "16 heads a group": (32, 2, 128, 48, [1, 1], [100, 47], True, 0),
    "64 heads a group": (64, 1, 64, 16, [1, 2], [65, 31], True, 0),
    "drafted tokens": (16, 2, 128, 64, [5, 1, 4], [513, 64, 4], True, 0),
    "a prompt": (6, 2, 64, 32, [70], [70], True, 0),
    "a chunk of a prompt": (8, 1, 128, 64, [45, 130], [300, 131], True, 0),
    "window": (4, 2, 128, 16, [1, 6, 40], [500, 90, 40], True, 33),
    "window of one": (2, 2, 64, 16, [3], [50], True, 1),
    "not causal": (4, 1, 64, 16, [3, 1], [50, 17], False, 0),
    "not causal, window": (4, 1, 128, 16, [3], [150], False, 20),
    "long": (8, 1, 128, 64, [1], [20011], True, 0),
    "long, several heads": (12, 4, 64, 128, [2], [6007], True, 0),
    "prompts of odd lengths": (12, 4, 64, 16, [129, 1, 300], [400, 900, 300], True, 0),
    "a prompt in a window": (8, 2, 128, 64, [300], [700], True, 100),
    "a prompt, not causal": (8, 4, 128, 32, [150], [333], False, 0),
}


def build(serve, case, seed=0, sizes=None):
    """Keys and values of `sizes(rng, tokens)` [tokens, 1, 1] times normal ones."""
    hq, hk, d, ps, new, kv, causal, window = CASES[case]
    rng = np.random.default_rng(seed)
    t = sum(new)
    held = [-(-x // ps) for x in kv]
    num = sum(held) + 3
    order = rng.permutation(num)
    table = np.full((len(new), max(max(held), 1)), num + 100, np.int32)  # what is never read may be anything
    cache = cache_of(serve, num, ps, hk, d, 0xFF)  # NaN codes in memory that is not written
    size = np.linspace(0.5, 2, hk)[:, None]
    keys, used = [], 0
    for b, n in enumerate(kv):
        table[b, :held[b]] = order[used:used + held[b]]
        used += held[b]
        slots = dev(table[b, np.arange(n) // ps].astype(np.int64) * ps + np.arange(n) % ps)
        k, v = (dev((rng.standard_normal((n, hk, d)) * size * (1 if sizes is None else sizes(rng, n, which))).astype(np.float32))
                for which in "kv")
        if n:
            cache.append(k, v, slots)
            cache.read(slots, k, v)
        keys.append((f64(k), f64(v)))
    q = dev(rng.standard_normal((max(t, 1), hq, d)), torch.bfloat16)
    cu = dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
    return cache, q, cu, dev(np.array(kv, np.int32)), dev(table), keys


def plans(cache, hq, requests):
    """Hints that lead to each of the kernels."""
    found = {}
    for max_q in (1, 2, 8, 32, 256, 10 ** 4, 10 ** 6):
        for max_kv in [0] + [2 ** i for i in range(5, 27)]:
            found.setdefault(cache.plan_kernel(hq, requests, max_q=max_q, max_kv=max_kv), (max_q, max_kv))
    return found


def check_all(case, cache, q, cu, kv_d, table, keys, scale=None):
    hq, hk, d, ps, new, kv, causal, window = CASES[case]
    kinds = plans(cache, hq, len(new))
    assert {n.split("<")[0] for n in kinds} == {"kv_attention_kernel", "kv_attention_team_kernel", "kv_attention_prompt_kernel"}
    assert len(kinds) >= 7, sorted(kinds)
    real = d ** -0.5 if scale is None else scale
    wants = [ref.attention(f64(q[at:at + n]), k, v, length, real, causal, window)
             for at, n, length, (k, v) in zip(np.cumsum([0] + new), new, kv, keys)]
    for name, (max_q, max_kv) in kinds.items():
        wide = torch.full((q.shape[0], hq + 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
        out, lse = wide[:, 1:1 + hq], torch.full((q.shape[0], hq), 7.0, device="cuda")
        for again in range(2):
            cache.attention(q, out, cu, kv_d, table, max_q=max_q, max_kv=max_kv, causal=causal, window=window, lse=lse, scale=scale)
            torch.cuda.synchronize()
            if again:
                assert torch.equal(out, first) and torch.equal(lse, first_lse), name  # noqa: F821
            first, first_lse = out.clone(), lse.clone()  # noqa: F841
        assert cache.status() == 0
        assert (wide[:, 0] == 7).all() and (wide[:, 1 + hq:] == 7).all()
        at = 0
        for n, length, (want, want_lse, mean, dots), (k, v) in zip(new, kv, wants, keys):
            got, empty = f64(lse[at:at + n]), np.isneginf(want_lse)
            assert np.array_equal(np.isneginf(got), empty), name
            assert (f64(out[at:at + n])[empty] == 0).all()
            tol = score_error(dots, d) + (length + 64) * U32 + 4 * U32 * np.abs(np.where(empty, 0, want_lse))
            assert (np.abs(got[~empty] - want_lse[~empty]) <= tol[~empty]).all(), name
            check_out(f64(out[at:at + n]), want, mean, dots, d, length, np.abs(v).max(initial=0.0))
            at += n
        assert (out[at:] == 7).all() and (lse[at:] == 7).all()


@pytest.mark.parametrize("case", sorted(CASES))
def test_attention_by_every_kernel(serve, case):
    check_all(case, *build(serve, case))


def wild(rng, n, which):
    """Sizes that change from block to block, of keys by 2^12, of values by 2^30: a block's exponent decides what its
    weights are worth."""
    span = 6 if which == "k" else 15
    return 2.0 ** np.repeat(rng.integers(-span, span, n // 16 + 1), 16)[:n, None, None]


@pytest.mark.parametrize("case", ["one token", "long", "drafted tokens", "prompts of odd lengths", "not causal", "window"])
def test_attention_with_exponents_that_differ(serve, case):
    built = build(serve, case, 3, wild)
    check_all(case, *built, scale=2.0 ** -8)


@pytest.mark.parametrize("case", ["drafted tokens", "a chunk of a prompt"])
@pytest.mark.parametrize("scale", [0.0, -0.1, 30.0, 1e-30])
def test_attention_scales(serve, case, scale):
    check_all(case, *build(serve, case), scale=scale)


def test_attention_in_graphs_and_on_streams(serve):
    case = "drafted tokens"
    cache, q, cu, kv_d, table, keys = build(serve, case)
    want = torch.empty_like(q)
    cache.attention(q, want, cu, kv_d, table, max_q=5, max_kv=513)
    side, out = torch.cuda.Stream(), torch.zeros_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        cache.attention(q, out, cu, kv_d, table, max_q=5, max_kv=513)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    k, v = torch.randn(3, 2, 128, device="cuda"), torch.randn(3, 2, 128, device="cuda")
    slots = dev(np.array([-1, -1, -1], np.int64))
    with torch.cuda.graph(graph):
        cache.append(k, v, slots)
        for plan in ((5, 513), (1, 2 ** 20), (10 ** 6, 2 ** 20)):
            cache.attention(q, out, cu, kv_d, table, max_q=plan[0], max_kv=plan[1])
        cache.attention(q, out, cu, kv_d, table, max_q=5, max_kv=513)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert cache.status() == 0


def test_pages_past_32_bits(serve):
    """A pool of 5 GB: offsets of pages do not fit 32 bits."""
    d, ps, hk = 128, 64, 8
    size = serve.kv8_page_bytes(ps, hk, d)
    num = 5 * 2 ** 30 // size
    cache = serve.KvCache8(torch.zeros(num, size, dtype=torch.uint8, device="cuda"), ps, hk, d)
    rng = np.random.default_rng(1)
    k, v = (dev(rng.standard_normal((70, hk, d)).astype(np.float32)) for _ in range(2))
    table = dev(np.array([[num - 1, num - 2]], np.int32))
    slots = dev(np.concatenate([(num - 1) * ps + np.arange(64), (num - 2) * ps + np.arange(6)]))
    cache.append(k, v, slots)
    cache.read(slots, k, v)
    assert k.abs().max() > 1
    q = dev(rng.standard_normal((1, 8, d)), torch.bfloat16)
    want, _, mean, dots = ref.attention(f64(q), f64(k), f64(v), 70, d ** -0.5, True, 0)
    for max_q, max_kv in ((1, 70), (1, 10 ** 7), (10 ** 5, 10 ** 5)):
        out = torch.zeros_like(q)
        cache.attention(q, out, dev(np.array([0, 1], np.int32)), dev(np.array([70], np.int32)), table, max_q=max_q, max_kv=max_kv)
        check_out(f64(out), want, mean, dots, d, 70, f64(v.abs().max()))
    assert cache.status() == 0


@pytest.mark.parametrize("gap", [1, 15, 16, 31, 33, 700])
def test_skipped_slots_do_not_come_between_neighbours(serve, gap):
    """Padding inside a batch: the tokens of a block on both sides of it are one run."""
    d, ps, hk = 64, 64, 2
    rng = np.random.default_rng(gap)
    cache = cache_of(serve, 40, ps, hk, d)
    pages = cache.pages.cpu().numpy().copy()
    for slots in (list(range(5, 9)) + [-1] * gap + list(range(9, 14)) + [10 ** 9] * gap + [14, 15, 16, 17],
                  [-1] * gap + list(range(100, 112)) + [-1] * gap,
                  sum(([s] + [-1] * gap for s in range(200, 235)), []),
                  list(range(300, 1800)) + [-1] * gap + list(range(1800, 1900))):
        x = dev(rng.standard_normal((len(slots), hk, d)) * 10.0 ** rng.uniform(-2, 2, (len(slots), 1, 1)), torch.bfloat16)
        cache.append(x, x * 2, dev(np.array(slots, np.int64)))
        more.append8(pages, ps, hk, d, f64(x), f64(x * 2), slots)
        assert np.array_equal(cache.pages.cpu().numpy(), pages)


def steps(span):
    """Sizes that change from block to block by 2^span at most: prompts take a tile's blocks in one unit up to 2^15."""
    return lambda rng, n, which: 2.0 ** np.repeat(rng.integers(0, span + 1, n // 16 + 1), 16)[:n, None, None]


@pytest.mark.parametrize("span", [1, 14, 15, 16, 17])
@pytest.mark.parametrize("case", ["prompts of odd lengths", "a chunk of a prompt", "a prompt in a window"])
def test_attention_with_exponents_about_as_far_apart_as_a_tile_takes(serve, case, span):
    check_all(case, *build(serve, case, span, steps(span)), scale=2.0 ** (-span - 3))
