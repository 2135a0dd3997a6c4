"""Attention of whole prompts on a GPU, against its definition in 64 bits."""
import numpy as np
import pytest

import serve_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# half steps: off by at most these relative to the value
U32, U16, U8 = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8
HALF = {torch.bfloat16: U8, torch.float16: U16}


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


def score_error(dots, d):
    """A score is a sum of d products in binary32, scaled; times log2(e), rounded, and exponentiated (2^-22 relative): an
    absolute error in the exponent."""
    return (d + 8) * 2 * U32 * dots + 2.0 ** -21


def attention(q, k, v, scale, causal, window):
    """As ref.attention, all queries of a head at once: out, lse, mean |v| under the weights, largest sum of |q_i k_i| |scale|."""
    n, hq, d = q.shape
    hk = k.shape[1]
    i, j = np.arange(n)[:, None], np.arange(n)[None]
    see = np.ones((n, n), bool)
    if causal:
        see &= j <= i
    if window:
        see &= j > i - window
    out, lse, mean, dots = np.zeros((n, hq, d)), np.zeros((n, hq)), np.zeros((n, hq, d)), np.zeros((n, hq))
    for h in range(hq):
        kh, vh = k[:, h * hk // hq], v[:, h * hk // hq]
        s = np.where(see, q[:, h] @ kh.T * scale, -np.inf)
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        total = p.sum(1, keepdims=True)
        out[:, h], lse[:, h] = p @ vh / total, (m + np.log(total))[:, 0]
        mean[:, h] = p @ np.abs(vh) / total
        dots[:, h] = np.where(see, np.abs(q[:, h]) @ np.abs(kh).T, 0).max(1) * abs(scale)
    return out, lse, mean, dots


def check(q, k, v, out, lse, cu, scale, causal, window):
    u, d = HALF[q.dtype], q.shape[2]
    for a, b in zip(cu, cu[1:]):
        n = b - a
        if n == 0:
            continue
        want, want_lse, mean, dots = attention(f64(q[a:b]), f64(k[a:b]), f64(v[a:b]), scale, causal, window)
        # a weight is rounded to the values' type; sums of n terms in binary32
        e = (u + 2 * score_error(dots, d) + (n + 64) * U32)[..., None]
        low = 2.0 ** -25 if q.dtype == torch.float16 else 0.0  # of results that are no normal binary16
        tol = u * np.abs(want) + (1 + u) * (e * mean + n * 2.0 ** -30 * np.abs(f64(v[a:b])).max()) + low + 1e-30
        got = f64(out[a:b])
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (bad.sum(), np.argwhere(bad)[:3], np.max(np.abs(got - want)[bad] / tol[bad]))
        tol = score_error(dots, d) + (n + 64) * U32 + 4 * U32 * np.abs(want_lse)
        assert (np.abs(f64(lse[a:b]) - want_lse) <= tol).all()


def build(rng, hq, hk, d, lengths, dtype, packed=True):
    t = sum(lengths)
    qkv = dev(rng.standard_normal((max(t, 1), hq + 2 * hk, d)), dtype)
    if packed:
        return qkv.split([hq, hk, hk], 1)
    return [x.contiguous() for x in qkv.split([hq, hk, hk], 1)]


CASES = {
    # name: hq, hk, d, lengths, causal, window
    "one token": (1, 1, 64, [1], True, 0),
    "one token of many heads": (64, 1, 128, [1], True, 0),
    "a few tokens": (8, 2, 128, [3, 1, 0, 7], True, 0),
    "groups of 7": (14, 2, 64, [70, 1, 33], True, 0),
    "groups of 5": (15, 3, 80, [100, 129], True, 0),
    "no groups": (3, 3, 128, [300, 5], True, 0),
    "narrow heads": (4, 2, 8, [50, 140], True, 0),
    "heads of 96": (4, 4, 96, [200], True, 0),
    "heads of 40": (6, 2, 40, [150], True, 0),
    "more heads than rows": (150, 1, 64, [21, 2], True, 0),
    "even more": (260, 1, 64, [5], True, 0),
    "tiles and one": (8, 1, 128, [128, 129, 127], True, 0),
    "a window": (8, 2, 64, [300, 40], True, 33),
    "a window of one": (4, 2, 128, [130], True, 1),
    "a window of tiles": (2, 1, 128, [700], True, 256),
    "not causal": (4, 2, 128, [200, 1, 77], False, 0),
    "not causal, a window": (4, 1, 64, [300], False, 50),
    "longer": (8, 1, 128, [1500], True, 0),
    "longer, not causal": (2, 2, 64, [1111], False, 0),
    "more segments than are dealt out": (16, 16, 64, [(11 * i) % 150 for i in range(120)], True, 0),
    "many of them and a window": (20, 20, 128, [(7 * i) % 40 for i in range(100)], True, 9),
    "many short": (4, 1, 64, [(7 * i) % 23 for i in range(300)], True, 0),
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", sorted(CASES))
def test_prompt(serve, case, dtype):
    hq, hk, d, lengths, causal, window = CASES[case]
    q, k, v = build(np.random.default_rng(1), hq, hk, d, lengths, dtype)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    prompts = serve.PromptAttention()
    for max_len in (1, 10 ** 6):
        wide = torch.full((q.shape[0] + 3, hq + 2, d), 7.0, dtype=dtype, device="cuda")
        out, lse = wide[:-3, 1:1 + hq], torch.full((q.shape[0], hq), 7.0, device="cuda")
        for again in range(2):
            prompts.attention(q, k, v, out, dev(cu), max_len=max_len, causal=causal, window=window, lse=lse)
            torch.cuda.synchronize()
            if again:
                assert torch.equal(out, first) and torch.equal(lse, first_lse)  # noqa: F821
            first, first_lse = out.clone(), lse.clone()  # noqa: F841
        assert prompts.status() == 0
        assert (wide[:, 0] == 7).all() and (wide[:, 1 + hq:] == 7).all() and (wide[-3:] == 7).all()
        assert (out[cu[-1]:] == 7).all() and (lse[cu[-1]:] == 7).all()
        check(q, k, v, out, lse, cu, d ** -0.5, causal, window)
    prompts.attention(q, k, v, out, dev(cu), max_len=max_len, causal=causal, window=window)  # no lse
    assert torch.equal(out, first)


@pytest.mark.parametrize("scale", [0.0, -0.2, 5.0, 1e-30])
def test_scales(serve, scale):
    q, k, v = build(np.random.default_rng(2), 4, 2, 64, [200, 30], torch.bfloat16)
    out, lse, prompts = torch.empty(230, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(230, 4, device="cuda"), serve.PromptAttention()
    prompts.attention(q, k, v, out, dev(np.array([0, 200, 230], np.int32)), max_len=200, scale=scale, lse=lse)
    check(q, k, v, out, lse, [0, 200, 230], scale, True, 0)


def test_strides_and_orders(serve):
    """Heads before tokens, and tensors that are not next to each other."""
    rng = np.random.default_rng(3)
    t, hq, hk, d = 170, 6, 3, 128
    q, k, v, out = (dev(rng.standard_normal((h, t, d)), torch.bfloat16).transpose(0, 1) for h in (hq, hk, hk, hq))
    lse, prompts = torch.empty(t, hq, device="cuda"), serve.PromptAttention()
    cu = [0, 100, 100, 170]
    prompts.attention(q, k, v, out, dev(np.array(cu, np.int32)), max_len=100, lse=lse)
    check(q, k, v, out, lse, cu, d ** -0.5, True, 0)


def test_rows_outside_the_prompts_stay(serve):
    """Tokens before the first and after the last prompt belong to none."""
    q, k, v = build(np.random.default_rng(4), 4, 2, 64, [90], torch.bfloat16)
    out, lse, prompts = torch.full((90, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((90, 4), 7.0, device="cuda"), serve.PromptAttention()
    prompts.attention(q, k, v, out, dev(np.array([10, 40, 77], np.int32)), max_len=40, lse=lse)
    check(q, k, v, out, lse, [10, 40, 77], 0.125, True, 0)
    assert (out[:10] == 7).all() and (out[77:] == 7).all() and (lse[:10] == 7).all() and (lse[77:] == 7).all()
    for bad in ([-5, 40, 10 ** 6], [50, 20, 90], [90, 0, 0], [2 ** 31 - 1, -2 ** 31, 3]):  # clamped, or rows several times
        prompts.attention(q, k, v, out, dev(np.array(bad, np.int32)), max_len=40, lse=lse)
    assert prompts.status() == 0
    prompts.attention(q, k, v, out, dev(np.array([-5, 40, 10 ** 6], np.int32)), max_len=40, lse=lse)
    check(q, k, v, out, lse, [0, 40, 90], 0.125, True, 0)


BAD = {"nan": float("nan"), "inf": float("inf"), "-inf": float("-inf")}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("what", sorted(BAD))
@pytest.mark.parametrize("max_len", [1, 10 ** 6])  # either kernel
@pytest.mark.parametrize("hq,hk,d,causal,window", [(4, 2, 64, True, 0), (2, 2, 128, True, 0), (8, 1, 128, True, 40), (4, 1, 64, False, 0)])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(serve, hq, hk, d, causal, window, max_len, what, dtype):
    lengths = [150, 300, 7]
    q, k, v = build(np.random.default_rng(5), hq, hk, d, lengths, dtype, packed=False)
    cu = [0, 150, 450, 457]
    prompts = serve.PromptAttention()
    out, lse = torch.empty_like(q), torch.empty(457, hq, device="cuda")
    run = lambda: prompts.attention(q, k, v, out, dev(np.array(cu, np.int32)), max_len=max_len, causal=causal, window=window, lse=lse)  # noqa: E731
    run()
    want, want_lse = out.clone(), lse.clone()
    places = [(0, 0, 3), (149, hk - 1, d - 1), (150 + 131, 0, 5), (150 + 131, 0, 6), (450, 0, 0), (456, hk - 1, 9)]
    for token, head, c in places:
        v[token, head, c] = BAD[what]
    run()
    torch.cuda.synchronize()
    assert torch.equal(lse, want_lse) and prompts.status() == 0
    hit = np.zeros(out.shape, bool)
    for token, head, c in places:
        b = np.searchsorted(cu, token, side="right") - 1
        for i in range(cu[b], cu[b + 1]):
            if (not causal or token <= i) and (not window or token > i - window):
                hit[i, head * (hq // hk):(head + 1) * (hq // hk), c] = True
    got, was = f64(out), f64(want)
    assert not np.isfinite(got[hit]).any()
    if what != "nan":
        assert (np.isnan(got[hit]) | (got[hit] == BAD[what])).all()
    assert np.array_equal(got[~hit], was[~hit])


@pytest.mark.parametrize("max_len", [1, 10 ** 6])
@pytest.mark.parametrize("what", sorted(BAD))
def test_values_that_are_not_finite_in_parts_that_are_joined(serve, what, max_len):
    """One prompt whose segments several CTAs share."""
    t, hq = 1800, 8
    q, k, v = build(np.random.default_rng(9), hq, 1, 128, [t], torch.bfloat16, packed=False)
    cu = dev(np.array([0, t], np.int32))
    prompts = serve.PromptAttention()
    out, lse, lse2 = torch.empty_like(q), torch.empty(t, hq, device="cuda"), torch.empty(t, hq, device="cuda")
    prompts.attention(q, k, v, out, cu, max_len=max_len, lse=lse)
    want = out.clone()
    places = [(1790, 3), (1660, 127), (900, 64), (897, 64), (130, 5)]  # in tiles that some rows see in part
    for token, c in places:
        v[token, 0, c] = BAD[what]
    prompts.attention(q, k, v, out, cu, max_len=max_len, lse=lse2)
    hit = torch.zeros_like(out, dtype=torch.bool)
    for token, c in places:
        hit[token:, :, c] = True
    assert not torch.isfinite(out[hit]).any() and torch.equal(out[~hit], want[~hit])
    assert torch.equal(lse, lse2) and prompts.status() == 0


@pytest.mark.parametrize("max_len", [1, 10 ** 6])
def test_keys_and_queries_that_are_not_finite(serve, max_len):
    """They make the rows that see the key, or have the query, NaN or infinite; no others change."""
    q, k, v = build(np.random.default_rng(6), 2, 1, 64, [200, 140], torch.bfloat16, packed=False)
    cu = dev(np.array([0, 200, 340], np.int32))
    prompts = serve.PromptAttention()
    out = torch.empty_like(q)
    prompts.attention(q, k, v, out, cu, max_len=max_len)
    want = out.clone()
    k[150, 0, 3], q[20, 1, 5] = float("nan"), float("inf")
    prompts.attention(q, k, v, out, cu, max_len=max_len)
    hit = torch.zeros(340, 2, dtype=torch.bool, device="cuda")
    hit[150:200] = True
    hit[20, 1] = True
    assert torch.equal(out[~hit], want[~hit]) and not torch.isfinite(out[150:200]).any()
    assert prompts.status() == 0


def test_graphs_streams_and_other_calls(serve):
    q, k, v = build(np.random.default_rng(7), 8, 2, 128, [400, 60], torch.bfloat16)
    cu = dev(np.array([0, 400, 460], np.int32))
    prompts = serve.PromptAttention()
    want, out = torch.empty(460, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(460, 8, 128, dtype=torch.bfloat16, device="cuda")
    prompts.attention(q, k, v, want, cu, max_len=400)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        prompts.attention(q, k, v, out, cu, max_len=400)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for max_len in (1, 10 ** 6, 1, 400):
            prompts.attention(q, k, v, out, cu, max_len=max_len)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    q2 = q.flip(0)
    prompts.attention(q2, k, v, out, cu, max_len=400)  # other inputs, the same workspace
    lse = torch.empty(460, 8, device="cuda")
    prompts.attention(q2, k, v, out, cu, max_len=400, lse=lse)
    check(q2, k, v, out, lse, [0, 400, 460], 128 ** -0.5, True, 0)
    assert prompts.status() == 0


@pytest.mark.parametrize("max_len", [1, 9001])
def test_a_long_prompt(serve, max_len):
    """More key tiles than CTAs, runs that end inside segments; against binary32 on the GPU, row by row."""
    rng = np.random.default_rng(8)
    t, hq, hk, d = 9001, 4, 1, 128
    q, k, v = build(rng, hq, hk, d, [t], torch.bfloat16)
    out, prompts = torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda"), serve.PromptAttention()
    lse = torch.empty(t, hq, device="cuda")
    prompts.attention(q, k, v, out, dev(np.array([0, t], np.int32)), max_len=max_len, lse=lse)
    assert prompts.status() == 0
    for i in [0, 1, 127, 128, 4999, 8191, 8192, 9000] + rng.integers(0, t, 40).tolist():
        s = q[i].double() @ k[:i + 1, 0].double().T * d ** -0.5
        p = torch.softmax(s, -1)
        want, mean = p @ v[:i + 1, 0].double(), p @ v[:i + 1, 0].double().abs()
        assert ((out[i].double() - want).abs() <= U8 * want.abs() + 1.01 * (U8 + 2e-5 + t * U32) * mean).all(), i
        assert ((lse[i].double() - torch.logsumexp(s, -1)).abs() <= 2e-5 + t * U32).all()
