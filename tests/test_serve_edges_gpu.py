"""Attention over the 4-bit cache where its kernels' numbers and paths reach
their ends, against plain references in 64 bits: through every kernel that a call
may be given."""
import numpy as np
import pytest

import serve_ref as ref
from test_serve_gpu import U8, U16, U32, _built, cache_of, dev, f64, plans, score_error, serve  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def one_request(serve, k, v, ps=64):  # noqa: F811
    """A cache that holds the keys and values k, v [kv, hk, d], their values as they are held, and its row of pages."""
    kv, hk, d = k.shape
    pages = -(-kv // ps)
    cache = cache_of(serve, pages, ps, hk, d)
    k, v, slots = dev(k.astype(np.float32)), dev(v.astype(np.float32)), torch.arange(kv, device="cuda")
    cache.append(k, v, slots)
    cache.read(slots, k, v)
    return cache, f64(k), f64(v), torch.arange(pages, dtype=torch.int32, device="cuda")[None]


def check_weights_far_below(serve, below, d, size):  # noqa: F811
    """One key outweighs each of the 131071 others, whose values are `size`, by 2^below; together they still count.  So many
    requests over the same pages that some have all keys in one run."""
    kv, hq, requests = 131072, 8, 160
    k, v = np.zeros((kv, 1, d)), np.full((kv, 1, d), size)
    k[0], v[0] = 1.0, 0.0
    cache, k, v, table = one_request(serve, k, v)
    q = dev(np.full((requests, hq, d), 1.0), torch.bfloat16)
    scale = below * np.log(2) / k[0].sum()
    want, want_lse, mean, dots = ref.attention(f64(q[:1]), k, v, kv, scale, True, 0)
    assert want[0, 0, 0] > 2.0 ** -13 * size
    # A weight is rounded to binary16, to 11 bits or, of small numbers, to a multiple of 2^-24: of weights taken at least
    # 2^7 times as large as they are against the largest, so within 2^-32 of that.
    lost = kv * 2.0 ** -32 * np.abs(v).max()
    tol = U8 * np.abs(want) + (1 + U8) * ((2 * U16 + 2 * score_error(dots, d) + (kv + 64) * U32)[..., None] * mean + lost)
    kinds = plans(cache, hq, requests)
    assert {n.split("<")[0] for n in kinds} == {"kv_attention_kernel", "kv_attention_team_kernel", "kv_attention_prompt_kernel"}
    for name, (max_q, max_kv) in kinds.items():
        out, lse = torch.empty_like(q), torch.empty(requests, hq, device="cuda")
        cache.attention(q, out, torch.arange(requests + 1, dtype=torch.int32, device="cuda"),
                        torch.full((requests,), kv, dtype=torch.int32, device="cuda"), table.repeat(requests, 1), max_q=max_q,
                        max_kv=max_kv, scale=scale, lse=lse)
        torch.cuda.synchronize()
        assert cache.status() == 0
        assert (np.abs(f64(out) - want) <= tol).all(), (name, f64(out).min(), f64(out).max(), want[0, 0, 0])
        assert (np.abs(f64(lse) - want_lse) <= score_error(dots, d) + (kv + 64) * U32 + 4 * U32 * np.abs(want_lse)).all(), name


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("below", [20.2, 24.6, 25.3, 28.0])
def test_many_weights_far_below_the_largest(serve, below, d):  # noqa: F811
    check_weights_far_below(serve, below, d, 1.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [20.0, 5000.0])
def test_many_weights_far_below_the_largest_over_large_values(serve, size, d):  # noqa: F811
    check_weights_far_below(serve, 25.3, d, size)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sizes", [(1e-3, 3.0, 20.0, 300.0, 12000.0), (12000.0, 40.0, 1e-3), (11.0, 13.0, 11.0, 26.0, 1.0)])
def test_values_whose_size_changes_along_the_keys(serve, sizes, d):  # noqa: F811
    """Stretches of a thousand keys with values of one size each; weights of like size."""
    rng = np.random.default_rng(8)
    each, hq = 1000, 8
    kv = each * len(sizes)
    v = rng.standard_normal((kv, 1, d)) * np.repeat(sizes, each)[:, None, None]
    cache, k, v, table = one_request(serve, rng.standard_normal((kv, 1, d)), np.clip(v, -12000, 12000))
    q = dev(rng.standard_normal((1, hq, d)), torch.bfloat16)
    want, want_lse, mean, dots = ref.attention(f64(q), k, v, kv, d ** -0.5, True, 0)
    # weights and their products: 11 bits, or multiples of 2^-24 of what is 2^7 times as large against the largest value
    lost = kv * 2.0 ** -32 * np.abs(v).max()
    tol = U8 * np.abs(want) + (1 + U8) * ((2 * U16 + 2 * score_error(dots, d) + (kv + 64) * U32)[..., None] * mean + lost)
    for name, (max_q, max_kv) in plans(cache, hq, 1).items():
        out, lse = torch.empty_like(q), torch.empty(1, hq, device="cuda")
        cache.attention(q, out, dev(np.array([0, 1], np.int32)), dev(np.array([kv], np.int32)), table, max_q=max_q, max_kv=max_kv, lse=lse)
        torch.cuda.synchronize()
        assert cache.status() == 0
        assert (np.abs(f64(out) - want) <= tol).all(), name
        assert (np.abs(f64(lse) - want_lse) <= score_error(dots, d) + (kv + 64) * U32 + 4 * U32 * np.abs(want_lse)).all(), name


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("code", [0.5, 1.5, 3.0])
def test_scores_of_keys_at_the_smallest_scales(serve, code, d):  # noqa: F811
    """Scales whose last bit is 2^-24, under queries that make scores of them: a score has every key's bits."""
    kv, hq = 300, 8
    s = (1025 + 4 * (np.arange(kv) % 250)) * 2.0 ** -24  # half of one, and 1 1/2, lie between two multiples of 2^-24
    k = np.repeat((code * s)[:, None], d, 1)
    k[:, ::32] = (6 * s)[:, None]
    v = np.random.default_rng(5).standard_normal((kv, 1, d))
    cache, held, v, table = one_request(serve, k[:, None], v)
    assert np.array_equal(held[:, 0], k)
    x = np.full((2, hq, d), 60000.0) * (1 + np.arange(hq) / 16)[None, :, None]
    x[..., ::32] = 0
    q = dev(x, torch.bfloat16)
    scale = 0.2 / code / d ** 0.5
    want, want_lse, mean, dots = ref.attention(f64(q), held, v, kv, scale, True, 0)
    assert dots.min() > 3
    for name, (max_q, max_kv) in plans(cache, hq, 1).items():
        out, lse = torch.empty_like(q), torch.empty(2, hq, device="cuda")
        cache.attention(q, out, dev(np.array([0, 2], np.int32)), dev(np.array([kv], np.int32)), table, max_q=max_q, max_kv=max_kv,
                        scale=scale, lse=lse)
        torch.cuda.synchronize()
        assert cache.status() == 0
        tol = score_error(dots, d) + (kv + 64) * U32 + 4 * U32 * np.abs(want_lse)
        assert (np.abs(f64(lse) - want_lse) <= tol).all(), (name, np.abs(f64(lse) - want_lse).max(), tol.min())
        e = (2 * U16 + 2 * score_error(dots, d) + (kv + 64) * U32)[..., None]
        assert (np.abs(f64(out) - want) <= U8 * np.abs(want) + (1 + U8) * e * mean).all(), name


@pytest.fixture(scope="module")
def impatient(tmp_path_factory):
    """The operators built with waits that run out at once."""
    import ctypes
    import subprocess

    from latency_barrier_free_gb300 import build_ext as be

    at = tmp_path_factory.mktemp("impatient")
    units = [f for f in be.SOURCES if f.startswith("serve")]
    run = [subprocess.Popen([be.nvcc(), *be.ARCH, *be.FLAGS, "-DRRA_ATTN_WAIT_NS=0", "-DRRA_ATTN_TRY_NS=0", "-c",
                             "%s/%s" % (be.CSRC, f), "-o", str(at / f) + ".o"], stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
           for f in units]
    assert [p.wait() for p in run] == [0] * len(units)
    subprocess.run([be.nvcc(), *be.ARCH, "-shared", "-cudart", "static", "-o", str(at / "lib.so"), *(str(at / f) + ".o" for f in units)],
                   check=True, stdout=subprocess.DEVNULL)
    lib = ctypes.CDLL(str(at / "lib.so"))
    lib.rra_kv_attention.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    return lib


def arguments(serve, cache, q, out, lse, cu, kv, table, max_q, max_kv):  # noqa: F811
    """The C structure of an attention call."""
    s = q.stride(0), q.stride(1), out.stride(0), out.stride(1)
    return serve._ATTN.pack(*serve._CACHE.unpack(cache._cache), q.data_ptr(), out.data_ptr(), lse.data_ptr(), cu.data_ptr(),
                            kv.data_ptr(), table.data_ptr(), cache._workspace.data_ptr(), *s, table.stride(0), q.shape[0],
                            q.shape[2] ** -0.5, kv.numel(), table.shape[1], q.shape[1], max_q, max_kv, 1, 0, 0)


@pytest.mark.parametrize("d", [64, 128])
def test_after_a_wait_ran_out_the_next_call_is_right(serve, impatient, d):  # noqa: F811
    """The call says that its waits ran out, and leaves the workspace as calls expect it."""
    from latency_barrier_free_gb300 import rra

    hq, hk, ps = 16, 2, 64
    new, kv = [40, 300, 7, 0] + [1] * 60, [5000, 9000, 300, 10] + [9000] * 60
    held = [-(-n // ps) for n in kv]
    cache = cache_of(serve, sum(held), ps, hk, d)
    table, used = torch.full((len(kv), max(held)), -1, dtype=torch.int32, device="cuda"), 0
    for b, n in enumerate(held):
        table[b, :n] = torch.arange(used, used + n, device="cuda")
        used += n
    gen = torch.Generator(device="cuda").manual_seed(4)
    for at in range(0, used * ps, 1 << 16):
        slots = torch.arange(at, min(at + (1 << 16), used * ps), device="cuda")
        cache.append(*(torch.randn(len(slots), hk, d, generator=gen, device="cuda") for _ in range(2)), slots)
    rng, flush = np.random.default_rng(12), torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    q = dev(rng.standard_normal((sum(new), hq, d)), torch.bfloat16)
    cu, kv_d = dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)), dev(np.array(kv, np.int32))
    head = cache._workspace[:4096].view(torch.int32)
    stream, ran_out = torch.cuda.current_stream().cuda_stream, set()
    for name, (max_q, max_kv) in plans(cache, hq, len(new)).items():
        want, lse = torch.empty_like(q), torch.empty(q.shape[0], hq, device="cuda")
        out, lse2 = torch.empty_like(want), torch.empty_like(lse)
        cache.attention(q, want, cu, kv_d, table, max_q=max_q, max_kv=max_kv, lse=lse)
        assert cache.status() == 0
        for way in ("the word", "reset()"):
            for _ in range(20):
                flush.fill_(0)  # copies come from memory, not from L2
                args = arguments(serve, cache, q, out, lse2, cu, kv_d, table, max_q, max_kv)
                assert impatient.rra_kv_attention(args, stream) == rra.OK
                if cache.status() != 0:
                    assert cache.status() == rra.ERR_TIMEOUT
                    ran_out.add(name)
                assert (head[1:] == 0).all(), name
            if way == "the word":
                head[0] = 0
            else:
                cache.reset()
            for _ in range(2):
                out.fill_(7.0)
                cache.attention(q, out, cu, kv_d, table, max_q=max_q, max_kv=max_kv, lse=lse2)
                assert cache.status() == 0 and torch.equal(out, want) and torch.equal(lse2, lse), name
    # the kernels that count arrivals in the workspace; small ones may find their few copies done
    assert {"kv_attention_kernel", "kv_attention_prompt_kernel"} <= {n.split("<")[0] for n in ran_out}, ran_out


@pytest.mark.parametrize("heads", [1, 8])
def test_steps_back_to_back_over_the_same_slots(serve, heads):  # noqa: F811
    """slot_map writes the slots that the write right behind it reads, step after step in one buffer, nothing in between."""
    n, ps, d, steps, width = 48, 16, 64, 60, 12
    pool = n * width
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    kv, table, cu, pos, short = i32(n), torch.full((n, width), -1, dtype=torch.int32, device="cuda"), i32(n + 1), i32(3 * n), i32(1)
    order = np.random.default_rng(2).permutation(pool).astype(np.int32)
    free, left = dev(order), torch.full((1,), pool, dtype=torch.int32, device="cuda")
    slots = torch.full((3 * n,), -1, dtype=torch.int64, device="cuda")
    cache = cache_of(serve, pool, ps, heads, d)
    rng = np.random.default_rng(3)
    new = rng.integers(0, 4, (steps, n)).astype(np.int32)
    new_d = dev(new)
    # the token at position p of request b has the value 2^((7 b + p) % 11) everywhere; its scale, a sixth of that, has 11 bits
    value = lambda b, p: 2.0 ** ((7 * b + p) % 11)  # noqa: E731
    x, at = np.zeros((steps, 3 * n, heads, d), np.float32), np.zeros(n, np.int64)
    for s in range(steps):
        b = np.repeat(np.arange(n), new[s])
        p = np.concatenate([np.arange(a, a + m) for a, m in zip(at, new[s])])
        x[s, :len(b)] = value(b, p)[:, None, None]
        at += new[s]
    x = dev(x, torch.bfloat16)
    torch.cuda.synchronize()
    for s in range(steps):
        serve.slot_map(kv, new_d[s], table, free, left, ps, kv_len=kv, cu_new=cu, slots=slots, positions=pos, free_left=left,
                       pages_short=short)
        cache.append(x[s], x[s], slots)
    torch.cuda.synchronize()
    assert kv.tolist() == at.tolist() and short.item() == 0 and at.max() <= width * ps
    rows = table.cpu().numpy()
    b = np.repeat(np.arange(n), at)
    p = np.concatenate([np.arange(m) for m in at])
    held = dev(rows[b, p // ps].astype(np.int64) * ps + p % ps)
    k, v = (torch.empty(len(b), heads, d, device="cuda") for _ in range(2))
    cache.read(held, k, v)
    want = np.broadcast_to(value(b, p)[:, None, None], k.shape)
    assert (np.abs(f64(k) - want) <= 2.0 ** -10 * want).all()
    assert torch.equal(k, v)


def test_a_gpu_that_is_not_the_current_one_is_refused(serve):  # noqa: F811
    """Said of the cache's GPU, before any tensor is looked at: one GPU is enough to see it."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = cache_of(serve, 4, 16, 2, 64)
    other, k, slots = cache._dev + 1, bf(3, 2, 64), torch.zeros(3, dtype=torch.int64, device="cuda")
    native = serve._native
    for call in (lambda: native.kv_append(cache._cache, other, k, k, slots, None),
                 lambda: native.kv_read(cache._cache, other, k, k, slots, None),
                 lambda: native.kv_attention(cache._cache, other, cache._workspace, bf(1, 2, 64), bf(1, 2, 64), i32(2), i32(1),
                                             i32(1, 4), 1, 1, 1.0, True, 0, None, None, 0)):
        with pytest.raises(ValueError, match="the current GPU is cuda:%d" % cache._dev):
            call()
    cache.append(k, k, slots)
    torch.cuda.synchronize()


def test_the_workspace_on_another_stream_than_its_own(serve):  # noqa: F811
    """Made behind other work on one stream, used on another, and gone before that work is done."""
    rng = np.random.default_rng(6)
    kv, hk, hq, d = 3000, 2, 8, 64
    cache, k, v, table = one_request(serve, rng.standard_normal((kv, hk, d)), rng.standard_normal((kv, hk, d)))
    q = dev(rng.standard_normal((30, hq, d)), torch.bfloat16)
    cu, kv_d = dev(np.array([0, 30], np.int32)), dev(np.array([kv], np.int32))
    away = torch.cuda.Stream()
    for max_q, max_kv in plans(cache, hq, 1).values():
        want, out = torch.empty_like(q), torch.zeros_like(q)
        cache.attention(q, want, cu, kv_d, table, max_q=max_q, max_kv=max_kv)
        size = cache._workspace.numel()
        dirt = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        del dirt
        torch.cuda._sleep(10 ** 7)
        fresh = serve.KvCache(cache.pages, cache.page_tokens, hk, d)
        with torch.cuda.stream(away):
            fresh.attention(q, out, cu, kv_d, table, max_q=max_q, max_kv=max_kv)
        away.synchronize()
        assert torch.equal(out, want) and fresh.status() == 0
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(away):
            torch.cuda._sleep(10 ** 7)
            fresh.attention(q, out, cu, kv_d, table, max_q=max_q, max_kv=max_kv)
        at = fresh._workspace.data_ptr()
        del fresh
        dirt = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(3)]
        assert at not in [x.data_ptr() for x in dirt]
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_status_of_work_on_another_stream(serve):  # noqa: F811
    cache = cache_of(serve, 1, 16, 1, 64)
    away = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(away):
        torch.cuda._sleep(10 ** 7)
        cache._workspace[:4].view(torch.int32).fill_(5)
    assert cache.status() == 5
    cache.reset()
    assert cache.status() == 0


def dense(q, k, v, scale, causal, window):
    """serve_ref.attention on the GPU: q [n, hq, d], k and v [kv, hk, d], float64.  Returns out, lse, mean |v| under the
    weights, and the largest sum of |q_i k_i| * |scale|, as numpy arrays."""
    n, hq, _ = q.shape
    kv, hk, _ = k.shape
    if kv == 0:
        return np.zeros(q.shape), np.full((n, hq), -np.inf), np.zeros(q.shape), np.zeros((n, hq))
    pos, key = kv - n + torch.arange(n, device="cuda")[:, None], torch.arange(kv, device="cuda")[None]
    see = torch.ones(n, kv, dtype=torch.bool, device="cuda")
    if causal:
        see &= key <= pos
    if window:
        see &= key > pos - window
    g = q.unflatten(1, (hk, -1))
    s = torch.einsum("nhgd,khd->nhgk", g, k) * scale
    dots = (torch.einsum("nhgd,khd->nhgk", g.abs(), k.abs()) * abs(scale)).masked_fill(~see[:, None, None], 0).amax(-1)
    s = s.masked_fill(~see[:, None, None], -torch.inf)
    lse = s.logsumexp(-1)
    p = (s - lse.masked_fill(lse == -torch.inf, 0.0)[..., None]).exp()
    out, mean = (torch.einsum("nhgk,khd->nhgd", p, x) for x in (v, v.abs()))
    return [x.flatten(1, 2).cpu().numpy() for x in (out, lse, mean, dots)]


WINDOWS = {
    # hq, hk, d, ps, requests, most new tokens, most keys, window, causal, kernels that the window leaves to choose from
    "many requests, several tiles": (16, 8, 64, 16, 200, 6, 2500, 700, True, {"8 rows", "16 rows", "128 rows", "256 rows", "1 CTA"}),
    "many requests, several tiles, heads of 128": (16, 8, 128, 48, 200, 6, 2500, 700, True,
                                                    {"8 rows", "16 rows", "128 rows", "256 rows", "1 CTA"}),
    "many requests, a narrow window": (16, 8, 64, 64, 400, 3, 900, 100, True, {"8 rows", "16 rows", "128 rows", "256 rows"}),
    "many requests, a narrow window, heads of 128": (16, 8, 128, 16, 400, 3, 900, 37, True,
                                                      {"8 rows", "16 rows", "128 rows", "256 rows"}),
    "prompts": (8, 2, 64, 64, 6, 600, 1500, 333, True, {"128 rows", "256 rows", "1 CTA", "2 CTAs", "4 CTAs"}),
    "prompts, heads of 128": (8, 2, 128, 16, 6, 600, 1500, 333, True, {"128 rows", "256 rows", "1 CTA", "2 CTAs", "4 CTAs"}),
    "prompts, not causal": (14, 2, 128, 64, 5, 300, 2200, 1000, False, {"128 rows", "256 rows", "1 CTA"}),
    "prompts, a window of one key": (8, 2, 64, 16, 6, 400, 900, 1, True, {"128 rows", "256 rows", "1 CTA"}),
}


@pytest.mark.parametrize("case", sorted(WINDOWS))
def test_windows_through_the_kernels_they_reach(serve, case):  # noqa: F811
    """The window cuts what is planned for, too: of the hints those are taken that lead to other kernels with it."""
    hq, hk, d, ps, n, most_new, most_kv, window, causal, want_kinds = WINDOWS[case]
    rng = np.random.default_rng(14)
    new = rng.integers(1, most_new + 1, n)
    kv = np.maximum(rng.integers(0, most_kv + 1, n), np.where(rng.random(n) < 0.8, new, 0))
    new[n // 2], kv[n // 3], kv[-1] = 0, 0, most_kv
    held = -(-kv // ps)
    num = int(held.sum())
    cache = cache_of(serve, num, ps, hk, d)
    table, order, used = np.full((n, max(held.max(), 1)), -1, np.int32), rng.permutation(num), 0
    for b in range(n):
        table[b, :held[b]] = order[used:used + held[b]]
        used += held[b]
    slots = np.concatenate([table[b, np.arange(kv[b]) // ps].astype(np.int64) * ps + np.arange(kv[b]) % ps for b in range(n)])
    gen = torch.Generator(device="cuda").manual_seed(7)
    k, v = (torch.randn(len(slots), hk, d, generator=gen, device="cuda") for _ in range(2))
    cache.append(k, v, dev(slots))
    cache.read(dev(slots), k, v)
    q = torch.randn(int(new.sum()), hq, d, generator=gen, device="cuda").bfloat16()
    cu, at = np.concatenate([[0], np.cumsum(new)]), np.concatenate([[0], np.cumsum(kv)])
    wants = [dense(q[cu[b]:cu[b + 1]].double(), k[at[b]:at[b + 1]].double(), v[at[b]:at[b + 1]].double(), d ** -0.5, causal, window)
             for b in range(n)]
    want, want_lse, mean, dots = (np.concatenate(x) for x in zip(*wants))
    length = np.repeat(np.minimum(kv, window + new), new)[:, None]
    kinds = {}
    for max_q in (1, 2, 8, 32, 64, 128, 256, 1024, 10 ** 4, 10 ** 6):
        for max_kv in [0] + [2 ** i for i in range(5, 27)]:
            name = cache.plan_kernel(hq, n, max_q=max_q, max_kv=max_kv, window=window)
            kinds.setdefault(name.split("<")[1][:-1], (max_q, max_kv))
    assert want_kinds <= set(kinds)
    empty = np.isneginf(want_lse)
    score = score_error(dots, d)
    tol = U8 * np.abs(want) + (1 + U8) * (2 * U16 + 2 * score + (length + 64) * U32)[..., None] * mean + 1e-30
    tol_lse = score + (length + 64) * U32 + 4 * U32 * np.abs(np.where(empty, 0, want_lse))
    cu_d, kv_d, table_d = dev(cu.astype(np.int32)), dev(kv.astype(np.int32)), dev(table)
    for name, (max_q, max_kv) in kinds.items():
        out, lse = torch.full_like(q, 7.0), torch.full((len(q), hq), 7.0, device="cuda")
        cache.attention(q, out, cu_d, kv_d, table_d, max_q=max_q, max_kv=max_kv, causal=causal, window=window, lse=lse)
        assert cache.status() == 0
        got, got_lse = f64(out), f64(lse)
        assert np.array_equal(np.isneginf(got_lse), empty) and (got[empty] == 0).all(), name
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (name, bad.sum())
        assert (np.abs(got_lse[~empty] - want_lse[~empty]) <= tol_lse[~empty]).all(), name


def test_query_ranges_that_hold_every_row_thousands_of_times(serve):  # noqa: F811
    """cu_q that goes up and down over 2^30 rows (of strides that overlap): more row tiles than 32 bits count.  The kernels for
    prompts leave at once."""
    hq, d, n, tokens = 64, 64, 4096, 2 ** 24 - 1
    cache = cache_of(serve, 1, 16, 1, d)
    x = torch.full((tokens * 8 + hq * d,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = x.clone()
    q, out = (z.as_strided((tokens, hq, d), (8, d, 1)) for z in (x, y))
    cu = dev(np.resize(np.array([0, tokens], np.int32), n + 1))
    kv, table = torch.ones(n, dtype=torch.int32, device="cuda"), torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    kinds = {name: hint for name, hint in plans(cache, hq, n).items() if name.startswith("kv_attention_prompt_kernel")}
    assert len(kinds) == 2
    for name, (max_q, max_kv) in kinds.items():
        assert cache.plan_kernel(hq, n, max_q=max_q, max_kv=max_kv) == name
        cache.attention(q, out, cu, kv, table, max_q=max_q, max_kv=max_kv)
        torch.cuda.synchronize()
        assert cache.status() == 0 and torch.equal(x, y)


@pytest.mark.parametrize("d", [64, 128])
def test_queries_with_one_element_far_above_the_rest(serve, d):  # noqa: F811
    """2^16 times the others, over a channel where no key has anything: the others keep all their bits."""
    rng = np.random.default_rng(15)
    kv, hq = 500, 8
    k = rng.standard_normal((kv, 1, d))
    k[..., 5] = 0
    cache, k, v, table = one_request(serve, k, rng.standard_normal((kv, 1, d)))
    x = rng.uniform(1, 2, (2, hq, d)) * np.where(rng.random((2, hq, d)) < 0.5, -1, 1) * 2.0 ** -16
    x[..., 5] = 1.5
    q = dev(x, torch.bfloat16)
    scale = 2.0 ** 16 / d ** 0.5
    want, want_lse, mean, dots = ref.attention(f64(q), k, v, kv, scale, True, 0)
    for name, (max_q, max_kv) in plans(cache, hq, 1).items():
        out, lse = torch.empty_like(q), torch.empty(2, hq, device="cuda")
        cache.attention(q, out, dev(np.array([0, 2], np.int32)), dev(np.array([kv], np.int32)), table, max_q=max_q, max_kv=max_kv,
                        scale=scale, lse=lse)
        assert cache.status() == 0
        e = (2 * U16 + 2 * score_error(dots, d) + (kv + 64) * U32)[..., None]
        assert (np.abs(f64(out) - want) <= U8 * np.abs(want) + (1 + U8) * e * mean).all(), name
        assert (np.abs(f64(lse) - want_lse) <= score_error(dots, d) + (kv + 64) * U32 + 4 * U32 * np.abs(want_lse)).all(), name


def test_every_kernel_from_a_graph_and_on_another_stream(serve):  # noqa: F811
    """The same bits as enqueued by itself; calls that follow each other over one workspace, replayed."""
    rng = np.random.default_rng(16)
    kv, hk, hq, d = 4000, 2, 16, 128
    cache, _, _, table = one_request(serve, rng.standard_normal((kv, hk, d)), rng.standard_normal((kv, hk, d)))
    q = dev(rng.standard_normal((200, hq, d)), torch.bfloat16)
    cu, kv_d = dev(np.array([0, 200], np.int32)), dev(np.array([kv], np.int32))
    away = torch.cuda.Stream()
    for name, (max_q, max_kv) in plans(cache, hq, 1).items():
        want, want_lse = torch.empty_like(q), torch.empty(200, hq, device="cuda")
        cache.attention(q, want, cu, kv_d, table, max_q=max_q, max_kv=max_kv, lse=want_lse)
        outs = [(torch.zeros_like(q), torch.zeros_like(want_lse)) for _ in range(3)]
        torch.cuda.synchronize()
        with torch.cuda.stream(away):
            cache.attention(q, outs[0][0], cu, kv_d, table, max_q=max_q, max_kv=max_kv, lse=outs[0][1])
        away.synchronize()
        assert torch.equal(outs[0][0], want) and torch.equal(outs[0][1], want_lse), name
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for out, lse in outs:
                cache.attention(q, out, cu, kv_d, table, max_q=max_q, max_kv=max_kv, lse=lse)
        for _ in range(2):
            for out, lse in outs:
                out.zero_(), lse.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(out, want) and torch.equal(lse, want_lse) for out, lse in outs), name
    assert cache.status() == 0
