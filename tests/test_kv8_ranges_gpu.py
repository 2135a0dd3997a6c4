"""The 8-bit cache at the ends of its ranges: exponents far apart, of values that a row does not see too, and scales and queries
that are very small or large."""
import ctypes

import numpy as np
import pytest

import serve_ref as ref
from test_kv8_gpu import U8, U16, U32, dev, f64, plans, score_error
from test_serve_edges_gpu import arguments, impatient  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def serve():
    from latency_barrier_free_gb300 import serve

    yield serve
    ref.leave_zeros()


def filled(serve, kind, k, v, ps, lengths):
    """A cache that holds k and v [tokens, heads, d] of requests of these lengths, its table, and what it holds."""
    hk, d = k.shape[1:]
    held = [-(-n // ps) for n in lengths]
    size = (serve.kv8_page_bytes if kind == 8 else serve.kv_page_bytes)(ps, hk, d)
    cache = (serve.KvCache8 if kind == 8 else serve.KvCache)(torch.full((sum(held), size), 0xFF, dtype=torch.uint8, device="cuda"), ps, hk, d)
    table, slots, used = np.full((len(lengths), max(held)), -1, np.int32), [], 0
    for b, n in enumerate(lengths):
        table[b, :held[b]] = used + np.arange(held[b])
        slots.append(used * ps + np.arange(n))
        used += held[b]
    slots = dev(np.concatenate(slots))
    k, v = dev(k.astype(np.float32)), dev(v.astype(np.float32))
    cache.append(k, v, slots)
    cache.read(slots, k, v)
    return cache, dev(table), f64(k), f64(v)


def formula(q, k, v, scale, causal, window):
    """out, lse, and of each row and channel: mean |v| under the weights, the largest |v| that the row sees; of each row, how far
    a score may be off.  The queries are the last."""
    n, kv, (hq, d), hk = len(q), len(k), q.shape[1:], k.shape[1]
    pos, j = kv - n + np.arange(n)[:, None], np.arange(kv)[None]
    see = np.broadcast_to(j <= pos if causal else j >= 0, (n, kv)) & (j > pos - window if window else j >= 0)
    out, mean, most = np.zeros((3, n, hq, d))
    lse, off = np.zeros((2, n, hq))
    for h in range(hq):
        kh, vh = k[:, h * hk // hq], v[:, h * hk // hq]
        s = np.where(see, q[:, h] @ kh.T * scale, -np.inf)
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        total = p.sum(1, keepdims=True)
        out[:, h], mean[:, h], lse[:, h] = p @ vh / total, p @ np.abs(vh) / total, (m + np.log(total))[:, 0]
        off[:, h] = score_error(np.where(see, np.abs(q[:, h]) @ np.abs(kh).T, 0).max(1) * abs(scale), d)
        # A query, scaled to [1, 2) by a power of two, is rounded to binary16: by half a step of 8 bits (none), but by up to
        # 2^-25, half of binary16's smallest number, where that is more; the power is at most the row's largest element.
        off[:, h] += 2.0 ** -25 * np.abs(q[:, h]).max(1) * np.where(see, np.abs(kh).sum(1), 0).max(1) * abs(scale)
        for i in range(n):
            most[i, h] = np.abs(vh[see[i]]).max(0)
    return out, lse, mean, most, off


def check(serve, kind, q, k, v, lengths, queries, scale, causal=True, window=0, ps=16):
    hq, d = q.shape[1:]
    cache, table, k, v = filled(serve, kind, k, v, ps, lengths)
    cu, kv_len = dev(np.cumsum([0] + queries).astype(np.int32)), dev(np.array(lengths, np.int32))
    q = dev(q.astype(np.float32)).bfloat16()
    ends, at = np.cumsum([0] + lengths), np.cumsum([0] + queries)
    wants = [formula(f64(q[a:b]), k[c:e], v[c:e], scale, causal, window) for a, b, c, e in zip(at, at[1:], ends, ends[1:])]
    for name, (max_q, max_kv) in plans(cache, hq, len(lengths)).items():
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        cache.attention(q, out, cu, kv_len, table, max_q=max_q, max_kv=max_kv, scale=scale, causal=causal, window=window, lse=lse)
        assert cache.status() == 0
        for (want, want_lse, mean, most, off), a, b, n in zip(wants, at, at[1:], lengths):
            # A weight is rounded to binary16, by half a step, or by 2^-25 where it is at least 2^7 times what it counts and its
            # block's unit at most 2^8 below that of the largest: 2^-24 of its value; the result to bfloat16.
            e = (U16 + 2 * off + (n + 64) * U32)[..., None]
            tol = U8 * np.abs(want) + (1 + U8) * (e * mean + n * 2.0 ** -24 * most) + 1e-30
            bad = ~(np.abs(f64(out[a:b]) - want) <= tol)
            assert not bad.any(), (name, bad.sum(), np.argwhere(bad)[:4], np.max(np.abs(f64(out[a:b]) - want)[bad] / tol[bad]))
            tol = off + (n + 64) * U32 + 4 * U32 * np.abs(want_lse)
            assert (np.abs(f64(lse[a:b]) - want_lse) <= tol).all(), name


@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 8, 1)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 100), (False, 0)])
@pytest.mark.parametrize("gap", [7, 8, 9, 20, 28, 32, 36, 40, 60])
def test_values_far_apart(serve, gap, causal, window, d, hq, hk):
    """Single values 2^gap times as large as the others, in one channel: rows that do not see them, and other channels, keep what
    they have."""
    rng = np.random.default_rng(gap)
    lengths, queries = [700, 33, 150], [230, 1, 150]
    k, v = rng.standard_normal((2, sum(lengths), hk, d))
    v *= 2.0 ** -20
    for token, channel in [(95, 3), (480, d - 1), (515, 8), (693, 0), (700 + 2, 5), (733 + 17, 1), (733 + 149, 2)]:
        v[token, :, channel] = 2.0 ** (gap - 20)
    check(serve, 8, rng.standard_normal((sum(queries), hq, d)), k, v, lengths, queries, d ** -0.5, causal, window)


@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 8, 1)])
def test_values_that_rise_and_fall(serve, d, hq, hk):
    """Blocks' units go up and down by up to 2^60, and so does which of them counts most."""
    rng = np.random.default_rng(1)
    lengths, queries = [1000, 400], [260, 2]
    k, v = rng.standard_normal((2, sum(lengths), hk, d))
    blocks = np.arange(sum(lengths)) // 16
    v *= (2.0 ** np.array([-20, 20, 0, -38, 22, -1, 21, -30, 7, 8, 0, 16, -16]))[blocks % 13][:, None, None]
    v *= np.where(rng.random((sum(lengths), 1, d)) < 0.9, 1, 0)
    check(serve, 8, rng.standard_normal((sum(queries), hq, d)), k, v, lengths, queries, 2.0)
    k *= np.exp2(rng.integers(-6, 6, len(blocks)))[:, None, None]
    check(serve, 8, rng.standard_normal((sum(queries), hq, d)), k, v, lengths, queries, 0.2, window=300)


@pytest.mark.parametrize("d", [64, 128])
def test_after_a_wait_ran_out_among_values_far_apart(serve, impatient, d):  # noqa: F811
    rng = np.random.default_rng(5)
    lengths, queries, hq, hk = [3000, 500], [400, 60], 8, 2
    k, v = rng.standard_normal((2, sum(lengths), hk, d))
    v *= (2.0 ** (np.arange(sum(lengths)) // 16 % 5 * 12 - 30))[:, None, None]
    cache, table, _, _ = filled(serve, 8, k, v, 64, lengths)
    cu, kv_len = dev(np.cumsum([0] + queries).astype(np.int32)), dev(np.array(lengths, np.int32))
    q = dev(rng.standard_normal((sum(queries), hq, d)).astype(np.float32)).bfloat16()
    impatient.rra_kv8_attention.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    flush, ran_out = torch.empty(1 << 28, dtype=torch.uint8, device="cuda"), 0
    for max_q, max_kv in plans(cache, hq, len(lengths)).values():
        want, lse = torch.empty_like(q), torch.empty(q.shape[0], hq, device="cuda")
        out, lse2 = torch.empty_like(want), torch.empty_like(lse)
        cache.attention(q, want, cu, kv_len, table, max_q=max_q, max_kv=max_kv, lse=lse)
        assert cache.status() == 0
        flush.zero_()
        args = arguments(serve, cache, q, out, lse2, cu, kv_len, table, max_q, max_kv)
        assert impatient.rra_kv8_attention(args, torch.cuda.current_stream().cuda_stream) == 0
        ran_out += cache.status() == 5
        assert (cache._workspace[:4096].view(torch.int32)[1:] == 0).all()
        cache.reset()
        cache.attention(q, out, cu, kv_len, table, max_q=max_q, max_kv=max_kv, lse=lse2)
        assert cache.status() == 0 and torch.equal(out, want) and torch.equal(lse, lse2)
    assert ran_out >= 5


@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 8, 1)])
@pytest.mark.parametrize("scale,by", [(1e-37, 1.0), (2.0 ** -60, 2.0 ** -60), (1.0, 2.0 ** -119), (-1e-38, 2.0 ** -10), (1e-30, 2.0 ** 20)])
def test_scores_that_are_next_to_nothing(serve, scale, by, d, hq, hk):
    """Keys of zero and of normal sizes: every score is about 0."""
    rng = np.random.default_rng(2)
    lengths, queries = [300, 20], [140, 20]
    k, v = rng.standard_normal((2, sum(lengths), hk, d))
    k[32:64] = 0
    k[100:] = 0
    check(serve, 8, rng.standard_normal((sum(queries), hq, d)) * by, k, v, lengths, queries, scale)


@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 8, 1)])
@pytest.mark.parametrize("scale,by", [(2.0 ** 40, 2.0 ** 60), (-(2.0 ** 50), 2.0 ** 50), (2.0 ** 100, 1.0), (2.0 ** 70, 2.0 ** 60), (2.0 ** 120, 2.0 ** 90)])
@pytest.mark.parametrize("kind", [8, 4])
def test_large_scales_over_scores_of_zero(serve, kind, scale, by, d, hq, hk):
    """Keys that are large where queries are 0: every score is 0, whatever it is scaled with."""
    rng = np.random.default_rng(3)
    lengths, queries = [300, 20], [140, 20]
    k, v = rng.standard_normal((2, sum(lengths), hk, d))
    k[..., 1:] = 0
    k *= 2.0 ** 39 if kind == 8 else 1.0
    q = rng.standard_normal((sum(queries), hq, d)) * by
    q[..., 0] = 0
    check(serve, kind, q, k, v, lengths, queries, scale)
