"""The decode-step operators on a GPU against plain references in 64 bits."""
import numpy as np
import pytest

import serve_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U16, U8, U32 = 2.0 ** -11, 2.0 ** -8, 2.0 ** -24  # unit roundoffs: binary16, bfloat16, binary32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    yield
    ref.leave_zeros()


@pytest.fixture(scope="module")
def serve():
    from latency_barrier_free_gb300 import serve

    return serve


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


# --------------------------------------------------------------- slot map --
def run_slot_map(serve, seq, new, table, free, count, ps, tokens, in_place=False, stream=None):
    n = len(seq)
    seq_d, table_d, free_d, count_d = dev(seq), dev(table), dev(free), dev(np.array([count], np.int32))
    i32 = lambda m: torch.full((m,), 77, dtype=torch.int32, device="cuda")  # noqa: E731
    kv = seq_d if in_place else i32(n)
    left = count_d if in_place else i32(1)
    cu, slots, pos, short = i32(n + 1), torch.full((tokens,), 77, dtype=torch.int64, device="cuda"), i32(tokens), i32(1)
    serve.slot_map(seq_d, dev(new), table_d, free_d, count_d, ps, kv_len=kv, cu_new=cu, slots=slots, positions=pos,
                   free_left=left, pages_short=short, stream=stream)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (kv, cu, slots, pos, left, short, table_d, free_d)]


def check_slot_map(serve, seq, new, table, free, count, ps, tokens, in_place=False):
    seq, new = np.asarray(seq, np.int32), np.asarray(new, np.int32)
    t2, f2 = table.copy(), free.copy()
    kv, cu, slots, pos, left, short = ref.slot_map(seq, new, t2, f2, count, ps, tokens)
    got = run_slot_map(serve, seq, new, table, free, count, ps, tokens, in_place)
    want = (kv, cu, slots, pos, [left], [short], t2, f2)
    for name, g, w in zip(("kv_len", "cu_new", "slots", "positions", "free_left", "pages_short", "table", "free"), got, want):
        assert np.array_equal(g, np.asarray(w).reshape(g.shape)), name
    return got


def make_pool(rng, seq, ps, width, pool):
    order = rng.permutation(pool).astype(np.int32)
    table = np.full((len(seq), width), -1, np.int32)
    used = 0
    for b, s in enumerate(seq):
        m = min(-(-max(s, 0) // ps), width)
        table[b, :m] = order[used:used + m]
        used += m
    free = np.zeros(pool, np.int32)
    free[:pool - used] = order[used:]
    return table, free, pool - used


@pytest.mark.parametrize("n,longest,ps,extra", [(1, 1, 1, 0), (1, 100, 16, 3), (7, 50, 16, 30), (33, 300, 64, 5000),
                                                (1000, 400, 16, 20000), (1025, 40, 7, 100), (4096, 70, 32, 40000)])
def test_slot_map_steps(serve, n, longest, ps, extra):
    rng = np.random.default_rng(n + ps)
    seq = rng.integers(0, longest + 1, n)
    new = np.where(rng.random(n) < 0.2, -rng.integers(1, 5, n), rng.integers(0, 4, n))
    new[rng.integers(0, n)] += extra
    width = -(-int((seq + np.maximum(new, 0)).max()) // ps) + 2
    pool = sum(-(-int(s + max(q, 0)) // ps) for s, q in zip(seq, new)) + 5
    table, free, count = make_pool(rng, seq, ps, width, pool)
    total = int(np.maximum(new, 0).sum())
    for tokens, in_place in ((total, False), (total + 13, True), (total // 2, False)):
        check_slot_map(serve, seq, new, table, free, count, ps, tokens, in_place)


def test_slot_map_short_pool_and_short_rows(serve):
    rng = np.random.default_rng(5)
    seq = np.array([30, 0, 17, 64, -3, 15], np.int32)
    table, free, count = make_pool(rng, seq, 16, 4, 12)
    got = check_slot_map(serve, seq, [100, 40, 1, 1, 20, -1], table, free, count, 16, 200)
    assert got[5][0] > 0 and (got[2] == -1).any()
    # entries that were never given do not go back to the stack
    table[2, :] = [-1, 99, 3, -1]
    check_slot_map(serve, seq, [0, 0, -1, -7, 0, 0], table, free, count, 16, 4)


def test_slot_map_nothing_to_do(serve):
    z = np.zeros(0, np.int32)
    got = run_slot_map(serve, z, z, np.zeros((0, 4), np.int32), np.arange(5, dtype=np.int32), 5, 16, 3)
    assert got[1].tolist() == [0] and got[2].tolist() == [-1] * 3 and got[4][0] == 5 and got[5][0] == 0
    got = run_slot_map(serve, np.array([3], np.int32), np.array([2], np.int32), np.zeros((1, 0), np.int32),
                       np.zeros(0, np.int32), 0, 16, 0)
    assert got[0].tolist() == [5] and got[5][0] == 0  # its second page was never due
    huge = np.full(3, 2 ** 31 - 1, np.int32)
    got = run_slot_map(serve, huge, huge, np.zeros((3, 2), np.int32), np.zeros(4, np.int32), 0, 16, 8)
    assert (got[2] == -1).all()


def test_slot_map_many_steps_keep_every_page(serve):
    """A serving run: requests arrive, grow, end; no page is ever lost or held twice."""
    rng = np.random.default_rng(11)
    n, ps, width, pool = 24, 16, 8, 110
    seq, table, free, count = np.zeros(n, np.int32), np.full((n, width), -1, np.int32), rng.permutation(pool).astype(np.int32), pool
    for step in range(40):
        new = np.where((seq > 0) & (rng.random(n) < 0.15), -1, np.where(seq == 0, rng.integers(0, 60, n), 1))
        new = np.where(seq + new > ps * width, -1, new).astype(np.int32)
        got = check_slot_map(serve, seq, new, table, free, count, ps, 64, in_place=bool(step % 2))
        seq, count, table, free = got[0].astype(np.int32), int(got[4][0]), got[6], got[7]
        if got[5][0]:
            break
        held = np.concatenate([table[b, :-(-seq[b] // ps)] for b in range(n)] + [free[:count]])
        assert np.array_equal(np.sort(held), np.arange(pool))


# ------------------------------------------------------ norms and rotation --
@pytest.mark.parametrize("t,hq,hk,d,rot,interleaved,dtype", [
    (1, 1, 1, 16, 16, False, "bf16"), (1, 8, 1, 128, 128, False, "bf16"), (5, 7, 3, 64, 64, True, "bf16"),
    (33, 4, 2, 80, 32, False, "fp32"), (17, 3, 1, 96, 96, True, "fp32"), (9, 5, 5, 256, 128, False, "bf16"),
    (4, 2, 2, 48, 48, False, "bf16"), (1000, 16, 3, 128, 64, True, "bf16"), (700, 24, 4, 128, 128, False, "fp32"),
    (11, 0, 3, 64, 64, False, "bf16"), (11, 3, 0, 64, 0, False, "fp32"), (600, 29, 8, 112, 112, False, "bf16")])
@pytest.mark.parametrize("case", ["plain", "packed", "in place", "no weight"])
def test_qk_norm_rope(serve, t, hq, hk, d, rot, interleaved, dtype, case):
    gen = torch.Generator().manual_seed(t + d)
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    most = 300
    x = (3 * torch.randn(t, hq + 2 * hk, d, generator=gen)).to(dt).cuda()
    x[0, :, :] *= 1e-4  # a small head: eps counts
    q, k = x[:, :hq], x[:, hq:hq + hk]
    if case == "plain":
        q, k = q.clone(), k.clone()
    wq = None if case == "no weight" else (1 + 0.3 * torch.randn(d, generator=gen)).to(dt).cuda()
    wk = (1 + 0.3 * torch.randn(d, generator=gen)).to(dt).cuda()
    pos = torch.randint(0, most, (t,), generator=gen).int()
    if t > 4:
        pos[2], pos[3] = most, -1  # outside the table
    angle = torch.arange(most)[:, None].double() * 10000.0 ** (-torch.arange(0, max(rot, 2), 2) / max(rot, 1)).double()
    cos, sin = (angle.cos().float().cuda(), angle.sin().float().cuda()) if rot else (None, None)
    eps = 1e-5
    args = (cos.double().cpu().numpy(), sin.double().cpu().numpy()) if rot else (None, None)
    want = [ref.norm_rope(f64(a), None if w is None else f64(w), *args, pos.numpy(), eps, interleaved)
            for a, w in ((q, wq), (k, wk))]
    if case == "in place":
        qo, ko, keep = q, k, x[:, hq + hk:].clone()
    else:
        wide = torch.full((t, hq + hk + 1, d), 7.0, dtype=dt, device="cuda")
        qo, ko = wide[:, :hq], wide[:, hq:hq + hk]
    if hq == 0:  # the first tensor says which GPU
        q, qo = x.new_empty(t, 0, d), x.new_empty(t, 0, d)
    serve.qk_norm_rope(q, k, wq, wk, cos, sin, pos.cuda(), qo, ko, eps=eps, interleaved=interleaved)
    torch.cuda.synchronize()
    # a sum of d squares, a reciprocal root (2 ulp), two products, a rotation of two terms: all in binary32
    rel = (d / 2 + 16) * U32
    for got, (y, size) in zip((qo, ko), want):
        g = f64(got)
        assert np.array_equal(np.isnan(g), np.isnan(y))
        y, g = np.nan_to_num(y), np.nan_to_num(g)
        tol = rel * size + (U8 * np.abs(y) + 2 * U8 * rel * size if dtype == "bf16" else 0) + 1e-30
        assert (np.abs(g - y) <= tol).all(), np.max(np.abs(g - y) - tol)
    if case == "in place":
        assert torch.equal(x[:, hq + hk:], keep)  # the values of the packed rows are untouched
    else:
        assert (wide[:, hq + hk:] == 7).all()


# ------------------------------------------------------------- the cache --
def cache_of(serve, num_pages, ps, hk, d, fill=0x7F):
    """Pages that were never written hold `fill`: as scales, NaN."""
    pages = torch.full((num_pages, serve.kv_page_bytes(ps, hk, d)), fill, dtype=torch.uint8, device="cuda")
    return serve.KvCache(pages, ps, hk, d)


@pytest.mark.parametrize("t,hk,d,ps,dtype", [(1, 1, 64, 16, "bf16"), (3, 2, 128, 16, "bf16"), (50, 3, 64, 48, "fp32"),
                                             (129, 8, 128, 64, "bf16"), (70, 5, 128, 128, "fp32"), (33, 1, 128, 4096, "fp32")])
def test_append_and_read(serve, t, hk, d, ps, dtype):
    rng = np.random.default_rng(t)
    num = -(-t // ps) + 2
    x = [rng.standard_normal((t, hk, d)).astype(np.float32) * 10.0 ** rng.integers(-6, 5, (t, hk, 1)) for _ in range(2)]
    x[0][0, 0, :8] = [0, -0.0, np.inf, -np.inf, np.nan, 1e-30, -5e-5, 65504]
    x[1][t // 2, 0, :] = 0
    # halfway between codes: the group's scale is exactly 1
    x[1][t - 1, 0, :32] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6] * 2
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    packed = torch.from_numpy(np.concatenate(x, 1)).to(dt).cuda()  # strided rows
    k, v = packed[:, :hk], packed[:, hk:]
    kn, vn = k.float().cpu().numpy(), v.float().cpu().numpy()
    slots = rng.permutation(num * ps)[:t].astype(np.int64)
    if t > 4:
        slots[1], slots[2], slots[3] = -1, num * ps, 2 ** 40
    cache = cache_of(serve, num, ps, hk, d, 0xA5)
    want = cache.pages.cpu().numpy()
    ref.write_pages(want, ps, hk, d, kn, vn, slots)
    cache.append(k, v, dev(slots))
    torch.cuda.synchronize()
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    back = torch.full((t, 2 * hk + 1, d), 7.0, dtype=dt, device="cuda")
    cache.read(dev(slots), back[:, :hk], back[:, hk:2 * hk])
    torch.cuda.synchronize()
    values = ref.read_pages(want, ps, hk, d, slots)
    for n, part in enumerate((back[:, :hk], back[:, hk:2 * hk])):
        assert torch.equal(part.cpu(), torch.from_numpy(values[n]).to(torch.float32).to(dt))
    assert (back[:, 2 * hk:] == 7).all()


def test_quantisation_error_is_half_a_step(serve):
    """Within the scale's range a value moves by at most half the step around it: scale/2 up to 4 scales, then 1 scale."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((64, 1, 128)).astype(np.float32)
    cache = cache_of(serve, 4, 16, 1, 128)
    k, slots = dev(x), torch.arange(64, device="cuda")
    cache.append(k, k, slots)
    got = torch.empty_like(k)
    cache.read(slots, got, torch.empty_like(k))
    torch.cuda.synchronize()
    g, y = x.reshape(-1, 32), got.cpu().numpy().reshape(-1, 32)
    s = np.abs(g).max(-1, keepdims=True) / 6
    step = np.where(np.abs(g) <= 2 * s, 0.25, np.where(np.abs(g) <= 4 * s, 0.5, 1.0)) * s
    assert (np.abs(g - y) <= step * (1 + 2.0 ** -9)).all()


@pytest.mark.parametrize("exponent", [-9, 0, 5])
def test_every_bfloat16_rounds_as_its_quotient(serve, exponent):
    """Every value of eight binades under every largest value of its group: midpoints of codes are among them."""
    binade = (1 + np.arange(128) / 128) * 2.0 ** exponent
    values = np.concatenate([binade * 2.0 ** -k for k in range(8)])
    rows = []
    for most in binade:
        x = values[values <= most]
        x = np.concatenate([x, -x])
        x = np.concatenate([x, np.zeros(-len(x) % 31)]).reshape(-1, 31)
        rows.append(np.concatenate([np.full((len(x), 1), most), x], 1))
    rows = np.concatenate(rows)
    rows = np.concatenate([rows, np.zeros((len(rows) % 2, 32))]).reshape(-1, 1, 64)
    cache = cache_of(serve, -(-len(rows) // 16), 16, 1, 64)
    k, slots = dev(rows, torch.bfloat16), torch.arange(len(rows), device="cuda")
    assert np.array_equal(f64(k), rows)
    cache.append(k, -k, slots)
    got = [torch.empty(rows.shape, device="cuda") for _ in range(2)]
    cache.read(slots, *got)
    want = ref.dequantise(*ref.quantise(rows.astype(np.float32)))
    for g, sign in zip(got, (1, -1)):
        assert np.array_equal(sign * f64(g), want)
        assert np.array_equal(np.signbit(f64(g)), np.signbit(sign * want))


def test_cache_beyond_4_gib(serve):
    """Pages whose byte offsets pass 32 bits."""
    hk, d, ps = 8, 128, 64
    num = 70000  # 5.2 GB
    cache = serve.KvCache(torch.zeros(num, serve.kv_page_bytes(ps, hk, d), dtype=torch.uint8, device="cuda"), ps, hk, d)
    rng = np.random.default_rng(4)
    kv = 150
    pages = np.array([num - 1, 3, num - 2], np.int32)
    slots = pages[np.arange(kv) // ps].astype(np.int64) * ps + np.arange(kv) % ps
    k = dev(rng.standard_normal((kv, hk, d)).astype(np.float32))
    v = dev(rng.standard_normal((kv, hk, d)).astype(np.float32))
    cache.append(k, v, dev(slots))
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    cache.read(dev(slots), kb, vb)
    q = dev(rng.standard_normal((1, hk, d)), torch.bfloat16)
    out = torch.empty_like(q)
    cache.attention(q, out, dev(np.array([0, 1], np.int32)), dev(np.array([kv], np.int32)), dev(pages[None]), max_q=1, max_kv=kv)
    torch.cuda.synchronize()
    codes, scales = ref.quantise(k.cpu().numpy())
    assert np.array_equal(f64(kb), ref.dequantise(codes, scales))
    want, _, mean, dots = ref.attention(f64(q), f64(kb), f64(vb), kv, d ** -0.5, True, 0)
    check_out(f64(out), want, mean, dots, d, kv)
    assert cache.status() == 0


# ------------------------------------------------------------- attention --
def score_error(dots, d):
    """A score is a sum of d products in binary32, scaled three times; times log2(e), rounded, and exponentiated
    (2^-22 relative): an absolute error in the exponent."""
    return (d + 8) * 2 * U32 * dots + 2.0 ** -21


def check_out(got, want, mean, dots, d, kv):
    # a weight is rounded to binary16, and so is its product with the scale; sums of kv terms in binary32
    e = (2 * U16 + 2 * score_error(dots, d) + (kv + 64) * U32)[..., None]
    tol = U8 * np.abs(want) + (1 + U8) * e * mean + 1e-30
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
    "a longer prompt": (16, 2, 128, 64, [257], [600], True, 0),
    "prompts of odd lengths": (12, 4, 64, 16, [129, 1, 300], [400, 900, 300], True, 0),
    "a prompt in a window": (8, 2, 128, 64, [300], [700], True, 100),
    "a prompt, not causal": (8, 4, 128, 32, [150], [333], False, 0),
}


def build(serve, case, seed=0, width_more=0):
    hq, hk, d, ps, new, kv, causal, window = CASES[case]
    rng = np.random.default_rng(seed)
    t = sum(new)
    held = [-(-x // ps) for x in kv]
    num = sum(held) + 3
    order = rng.permutation(num)
    width = max(max(held), 1) + width_more
    table = np.full((len(new), width), num + 100, np.int32)  # what is never read may be anything
    cache = cache_of(serve, num, ps, hk, d)
    size = np.linspace(0.5, 2, hk)[:, None]
    keys, used = [], 0
    for b, n in enumerate(kv):
        table[b, :held[b]] = order[used:used + held[b]]
        used += held[b]
        slots = dev(table[b, np.arange(n) // ps].astype(np.int64) * ps + np.arange(n) % ps)
        k, v = (dev((rng.standard_normal((n, hk, d)) * size).astype(np.float32)) for _ in range(2))
        if n:
            cache.append(k, v, slots)
            cache.read(slots, k, v)
        keys.append((f64(k), f64(v)))
    q = dev(rng.standard_normal((max(t, 1), hq, d)), torch.bfloat16)
    cu = dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
    return cache, q, cu, dev(np.array(kv, np.int32)), table, keys


@pytest.mark.parametrize("case", sorted(CASES))
def test_attention(serve, case):
    hq, hk, d, ps, new, kv, causal, window = CASES[case]
    cache, q, cu, kv_d, table, keys = build(serve, case)
    t = sum(new)
    wide = torch.full((q.shape[0], hq + 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
    out, lse = wide[:, 1:1 + hq], torch.full((q.shape[0], hq), 7.0, device="cuda")
    kw = dict(max_q=max(new), max_kv=max(kv), causal=causal, window=window, lse=lse)
    cache.attention(q, out, cu, kv_d, dev(table), **kw)
    torch.cuda.synchronize()
    assert cache.status() == 0
    assert (wide[:, 0] == 7).all() and (wide[:, 1 + hq:] == 7).all() and (out[t:] == 7).all()
    first, first_lse = out.clone(), lse.clone()
    at = 0
    for n, length, (k, v) in zip(new, kv, keys):
        want, want_lse, mean, dots = ref.attention(f64(q[at:at + n]), k, v, length, d ** -0.5, causal, window)
        check_out(f64(out[at:at + n]), want, mean, dots, d, length)
        got = f64(lse[at:at + n])
        empty = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(got), empty) and (f64(out[at:at + n])[empty] == 0).all()
        tol = score_error(dots, d) + (length + 64) * U32 + 4 * U32 * np.abs(np.where(empty, 0, want_lse))
        assert (np.abs(got - want_lse)[~empty] <= tol[~empty]).all()
        at += n
    # the same bits again, whatever the plan was told, on another stream, and replayed from a graph
    for hint_q, hint_kv in ((max(new), max(kv)), (max(new), 1)):
        wide.fill_(7.0)
        cache.attention(q, out, cu, kv_d, dev(table), **dict(kw, max_q=hint_q, max_kv=hint_kv))
        torch.cuda.synchronize()
        check_same = torch.equal(out, first) and torch.equal(lse, first_lse)
        assert check_same or hint_kv != max(kv)
        assert (out.float() - first.float()).abs().max() <= 0.02 * max(1.0, first.float().abs().max())


def plans(cache, hq, requests):
    """Hints that lead to each of the kernels."""
    found = {}
    for max_q in (1, 2, 8, 32, 256, 10 ** 4, 10 ** 6):
        for max_kv in [0] + [2 ** i for i in range(5, 27)]:
            found.setdefault(cache.plan_kernel(hq, requests, max_q=max_q, max_kv=max_kv), (max_q, max_kv))
    return found


@pytest.mark.parametrize("case", sorted(CASES))
def test_every_kernel_is_right_for_every_call(serve, case):
    """What the caller expects decides which kernel runs, not what it computes."""
    hq, hk, d, ps, new, kv, causal, window = CASES[case]
    cache, q, cu, kv_d, table, keys = build(serve, case)
    kinds = plans(cache, hq, len(new))
    assert {n.split("<")[0] for n in kinds} == {"kv_attention_kernel", "kv_attention_team_kernel", "kv_attention_prompt_kernel"}
    assert len(kinds) >= 7, sorted(kinds)
    wants = [ref.attention(f64(q[at:at + n]), k, v, length, d ** -0.5, causal, window)
             for at, n, length, (k, v) in zip(np.cumsum([0] + new), new, kv, keys)]
    for name, (max_q, max_kv) in kinds.items():
        out, lse = torch.full_like(q, 7.0), torch.full((q.shape[0], hq), 7.0, device="cuda")
        cache.attention(q, out, cu, kv_d, dev(table), max_q=max_q, max_kv=max_kv, causal=causal, window=window, lse=lse)
        torch.cuda.synchronize()
        at = 0
        for n, length, (want, want_lse, mean, dots) in zip(new, kv, wants):
            check_out(f64(out[at:at + n]), want, mean, dots, d, length)
            got, empty = f64(lse[at:at + n]), np.isneginf(want_lse)
            assert np.array_equal(np.isneginf(got), empty), name
            tol = score_error(dots, d) + (length + 64) * U32 + 4 * U32 * np.abs(np.where(empty, 0, want_lse))
            assert (np.abs(got[~empty] - want_lse[~empty]) <= tol[~empty]).all(), name
            at += n
        assert (out[at:] == 7).all()
    assert cache.status() == 0


@pytest.mark.parametrize("case", ["a chunk of a prompt", "drafted tokens", "a longer prompt"])
def test_attention_hints_do_not_decide_what_is_computed(serve, case):
    hq, hk, d, ps, new, kv, causal, window = CASES[case]
    cache, q, cu, kv_d, table, keys = build(serve, case)
    for max_q, max_kv in ((0, 0), (1, 1), (10 ** 6, 10 ** 6), (max(new), 1), (1, max(kv))):
        out = torch.full_like(q, 7.0)
        cache.attention(q, out, cu, kv_d, dev(table), max_q=max_q, max_kv=max_kv)
        torch.cuda.synchronize()
        at = 0
        for n, length, (k, v) in zip(new, kv, keys):
            want, _, mean, dots = ref.attention(f64(q[at:at + n]), k, v, length, d ** -0.5, causal, window)
            check_out(f64(out[at:at + n]), want, mean, dots, d, length)
            at += n
    assert cache.status() == 0


def test_attention_in_a_graph_and_on_another_stream(serve):
    case = "drafted tokens"
    hq, hk, d, ps, new, kv, causal, window = CASES[case]
    cache, q, cu, kv_d, table, keys = build(serve, case)
    table = dev(table)
    want = torch.empty_like(q)
    cache.attention(q, want, cu, kv_d, table, max_q=5, max_kv=513)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.zeros_like(q)
    with torch.cuda.stream(side):
        cache.attention(q, out, cu, kv_d, table, max_q=5, max_kv=513)
    side.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            cache.attention(q, out, cu, kv_d, table, max_q=5, max_kv=513)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("case", ["one token", "a chunk of a prompt", "a longer prompt"])
def test_attention_with_pages_that_are_not_there(serve, case):
    """Keys in pages outside the cache are not seen; lengths past the table are cut."""
    hq, hk, d, ps, new, kv, causal, window = CASES[case]
    cache, q, cu, kv_d, table, keys = build(serve, case)
    table[0, 1] = -1
    held = -(-kv[0] // ps)
    if held > 3:
        table[0, 3] = 2 ** 31 - 1
    out = torch.empty_like(q)
    cache.attention(q, out, cu, kv_d, dev(table), max_q=max(new), max_kv=max(kv))
    torch.cuda.synchronize()
    page = np.arange(kv[0]) // ps
    want, _, mean, dots = ref.attention(f64(q[:new[0]]), *keys[0], kv[0], d ** -0.5, True, 0, (page != 1) & (page != 3))
    check_out(f64(out[:new[0]]), want, mean, dots, d, kv[0])
    assert cache.status() == 0
    # a length beyond the row of pages: as if it ended there
    short = dev(table[:, :1])
    cache.attention(q, out, cu, dev(np.full(len(new), 10 ** 9, np.int32)), short, max_q=max(new), max_kv=max(kv))
    torch.cuda.synchronize()
    n = min(new[0], 16)
    k, v = (x[:ps] for x in keys[0])
    want, _, mean, dots = ref.attention(f64(q[:new[0]]), k, v, ps, d ** -0.5, True, 0)
    check_out(f64(out[:n]), want[:n], mean[:n], dots[:n], d, ps)
    # query ranges outside the tensor are cut, too
    cache.attention(q, out, dev(np.arange(len(new) + 1, dtype=np.int32) * 10 ** 6 - 5), kv_d, dev(table), max_q=1, max_kv=1)
    torch.cuda.synchronize()
    assert cache.status() == 0


@pytest.mark.parametrize("new", [1, 200])
@pytest.mark.parametrize("size", [1e-30, 1e-3, 300.0, 1e20])
def test_attention_of_queries_of_any_size(serve, size, new):
    rng = np.random.default_rng(9)
    hq, hk, d, ps, kv = 8, 2, 128, 16, 210
    cache = cache_of(serve, 16, ps, hk, d)
    k, v = (dev(rng.standard_normal((kv, hk, d)).astype(np.float32)) for _ in range(2))
    slots = torch.arange(kv, device="cuda")
    cache.append(k, v, slots)
    cache.read(slots, k, v)
    q = dev(rng.standard_normal((new, hq, d)) * size, torch.bfloat16)
    out = torch.empty_like(q)
    table = torch.arange(16, dtype=torch.int32, device="cuda")[None]
    for scale in (d ** -0.5, -0.1, 0.0):
        cache.attention(q, out, dev(np.array([0, new], np.int32)), dev(np.array([kv], np.int32)), table, max_q=new, max_kv=kv,
                        scale=scale)
        torch.cuda.synchronize()
        want, _, mean, dots = ref.attention(f64(q), f64(k), f64(v), kv, scale, True, 0)
        got = f64(out)
        sharp = dots > 1e3  # scores so far apart that rounding decides between close ones: only finiteness is claimed
        assert np.isfinite(got).all()
        check_out(np.where(sharp[..., None], want, got), want, mean, dots, d, kv)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("values", ["small", "small, then large", "large"])
def test_weights_far_below_one(serve, d, values):
    """Thousands of keys in one run whose weights are far below the largest: weight times scale keeps its bits."""
    rng = np.random.default_rng(31)
    hq, hk, ps, kv = 8, 1, 64, 9000
    cache = cache_of(serve, -(-kv // ps), ps, hk, d)
    size = np.full((kv, 1, 1), 2e-4)
    if values != "small":
        size[0 if values == "large" else 5000:] = 3000.0
    k, v = (dev((rng.standard_normal((kv, hk, d)) * x).astype(np.float32)) for x in (1.0, size))
    slots = torch.arange(kv, device="cuda")
    cache.append(k, v, slots)
    cache.read(slots, k, v)
    q = dev(rng.standard_normal((1, hq, d)) * 4, torch.bfloat16)
    table = torch.arange(-(-kv // ps), dtype=torch.int32, device="cuda")[None]
    want, want_lse, mean, dots = ref.attention(f64(q), f64(k), f64(v), kv, d ** -0.5, True, 0)
    for name, (max_q, max_kv) in plans(cache, hq, 1).items():
        out, lse = torch.empty_like(q), torch.empty(1, hq, device="cuda")
        cache.attention(q, out, dev(np.array([0, 1], np.int32)), dev(np.array([kv], np.int32)), table, max_q=max_q, max_kv=max_kv, lse=lse)
        torch.cuda.synchronize()
        check_out(f64(out), want, mean, dots, d, kv)
        assert (np.abs(f64(lse) - want_lse) <= score_error(dots, d) + (kv + 64) * U32 + 4 * U32 * np.abs(want_lse)).all(), name


@pytest.mark.parametrize("d,hk,group", [(128, 3, 2), (64, 2, 7)])
def test_large_queries_that_see_no_key(serve, d, hk, group):
    """Rows before the first key, in segments that warps and CTAs share, where the scale of a row is above 1."""
    hq, ps, new, kv = hk * group, 48, [0, 50, 402], [1, 2, 402]
    rng = np.random.default_rng(21)
    num = sum(-(-n // ps) for n in kv)
    cache = cache_of(serve, num, ps, hk, d)
    table = np.zeros((3, -(-max(kv) // ps)), np.int32)
    keys, used = [], 0
    for b, n in enumerate(kv):
        held = -(-n // ps)
        table[b, :held] = np.arange(used, used + held)
        used += held
        slots = dev(table[b, np.arange(n) // ps].astype(np.int64) * ps + np.arange(n) % ps)
        k, v = (dev(rng.standard_normal((n, hk, d)).astype(np.float32) * 0.01) for _ in range(2))
        cache.append(k, v, slots)
        cache.read(slots, k, v)
        keys.append((f64(k), f64(v)))
    q = dev(rng.standard_normal((sum(new), hq, d)) * 100, torch.bfloat16)
    cu = dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
    for name, (max_q, max_kv) in plans(cache, hq, 3).items():
        out, lse = torch.full_like(q, 7.0), torch.full((q.shape[0], hq), 7.0, device="cuda")
        cache.attention(q, out, cu, dev(np.array(kv, np.int32)), dev(table), max_q=max_q, max_kv=max_kv, lse=lse)
        torch.cuda.synchronize()
        assert cache.status() == 0
        for b in (1, 2):
            rows = slice(int(cu[b]), int(cu[b + 1]))
            want, want_lse, mean, dots = ref.attention(f64(q[rows]), *keys[b], kv[b], d ** -0.5, True, 0)
            empty = np.isneginf(want_lse)
            assert empty[:48].all() == (b == 1)
            assert np.array_equal(np.isneginf(f64(lse[rows])), empty), name
            assert (f64(out[rows])[empty] == 0).all(), name
            check_out(f64(out[rows]), want, mean, dots, d, kv[b])


def test_attention_nan_query_stays_in_its_row(serve):
    for case in ("drafted tokens", "a longer prompt"):
        hq, hk, d, ps, new, kv, causal, window = CASES[case]
        cache, q, cu, kv_d, table, keys = build(serve, case)
        want, _, mean, dots = ref.attention(f64(q[:new[0]]), *keys[0], kv[0], d ** -0.5, causal, window)
        out = torch.empty_like(q)
        q[1, 3, 5] = float("nan")
        q[2, 0, 0] = float("inf")
        cache.attention(q, out, cu, kv_d, dev(table), max_q=max(new), max_kv=max(kv))
        torch.cuda.synchronize()
        assert out[1, 3].isnan().all() and out[2, 0].isnan().all()
        got = f64(out[:new[0]])
        got[1, 3], got[2, 0] = want[1, 3], want[2, 0]
        check_out(got, want, mean, dots, d, kv[0])


@pytest.mark.parametrize("max_q", [1, 64])
def test_attention_of_many_requests(serve, max_q):
    """The most requests of one call, most of them tiny."""
    n, hq, hk, d, ps = 4096, 4, 2, 64, 16
    rng = np.random.default_rng(3)
    kv = rng.integers(0, 40, n)
    kv[17] = 3000
    held = -(-kv // ps)
    num = int(held.sum())
    cache = cache_of(serve, num, ps, hk, d)
    table = np.full((n, held.max()), -1, np.int32)
    used = 0
    for b in range(n):
        table[b, :held[b]] = np.arange(used, used + held[b])
        used += held[b]
    slots = np.concatenate([table[b, np.arange(kv[b]) // ps].astype(np.int64) * ps + np.arange(kv[b]) % ps for b in range(n)])
    k, v = (dev(rng.standard_normal((len(slots), hk, d)).astype(np.float32)) for _ in range(2))
    cache.append(k, v, dev(slots))
    cache.read(dev(slots), k, v)
    q = dev(rng.standard_normal((n, hq, d)), torch.bfloat16)
    out = torch.empty_like(q)
    cache.attention(q, out, dev(np.arange(n + 1, dtype=np.int32)), dev(kv.astype(np.int32)), dev(table), max_q=max_q, max_kv=3000)
    torch.cuda.synchronize()
    assert cache.status() == 0
    at = np.concatenate([[0], np.cumsum(kv)])
    kn, vn, qn, got = f64(k), f64(v), f64(q), f64(out)
    for b in list(range(0, n, 37)) + [17, n - 1]:
        want, _, mean, dots = ref.attention(qn[b:b + 1], kn[at[b]:at[b + 1]], vn[at[b]:at[b + 1]], int(kv[b]), d ** -0.5, True, 0)
        check_out(got[b:b + 1], want, mean, dots, d, int(kv[b]))


# -------------------------------------------------- the binding's refusals --
def test_binding_refuses_what_does_not_fit(serve):
    """Wrong types, shapes, strides and places raise before anything is launched."""
    from latency_barrier_free_gb300 import rra

    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    cache = cache_of(serve, 4, 16, 2, 64)
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    good = [bf(3, 2, 64), bf(3, 2, 64), slots]
    cache.append(*good)
    for n, bad in ((0, bf(3, 2, 32)), (0, bf(2, 2, 64)), (1, bf(3, 2, 64).float()), (0, bf(3, 2, 64).cpu()),
                   (0, bf(3, 64, 2).transpose(1, 2)), (2, i32(3)), (2, slots.cpu()), (1, bf(6, 64)), (2, slots.expand(3, 3)[:, 1])):
        args = list(good)
        args[n] = bad
        with pytest.raises(ValueError):
            cache.append(*args)
    with pytest.raises(TypeError):
        cache.append(bf(3, 2, 64).double(), bf(3, 2, 64), slots)
    with pytest.raises(rra.RraError):  # a stride that is no multiple of 16 bytes
        cache.append(bf(3, 2 * 64 + 1)[:, :128].view(3, 2, 64), good[1], slots)
    q, table, cu, kv = bf(2, 4, 64), i32(2, 3), i32(3), i32(2)
    kw = dict(max_q=1, max_kv=8)
    cache.attention(q, bf(2, 4, 64), cu, kv, table, **kw)
    for args, more in (((q, bf(2, 4, 32), cu, kv, table), {}), ((bf(2, 3, 64), bf(2, 3, 64), cu, kv, table), {}),
                       ((q, q.float(), cu, kv, table), {}), ((q, bf(2, 4, 64), i32(2), kv, table), {}),
                       ((q, bf(2, 4, 64), cu, kv, i32(3, 3)), {}), ((q, bf(2, 4, 64), cu, kv, table.t()), {}),
                       ((q, bf(2, 4, 64), cu, kv.long(), table), {}), ((q, bf(2, 4, 64), cu, kv, table), {"lse": bf(2, 4)}),
                       ((q, bf(2, 4, 64), cu, kv, table), {"lse": torch.zeros(7, device="cuda")})):
        with pytest.raises(ValueError):
            cache.attention(*args, **kw, **more)
    with pytest.raises(rra.RraError):
        cache.attention(q, bf(2, 4, 64), cu, kv, table, max_q=-1, max_kv=8)
    k, c = bf(2, 1, 64), torch.zeros(9, 32, device="cuda")
    ok = [q, k, None, bf(64), c, c, i32(2), bf(2, 4, 64), bf(2, 1, 64)]
    serve.qk_norm_rope(*ok)
    for n, bad in ((1, bf(3, 1, 64)), (2, bf(63)), (3, bf(64).float()), (4, torch.zeros(8, 32, device="cuda")), (6, i32(1)),
                   (6, slots), (7, bf(2, 3, 64)), (8, bf(2, 1, 64).cpu()), (5, c.cpu())):
        args = list(ok)
        args[n] = bad
        with pytest.raises(ValueError):
            serve.qk_norm_rope(*args)
    with pytest.raises(ValueError):
        serve.KvCache(torch.zeros(100, dtype=torch.uint8, device="cuda"), 16, 2, 64)
    assert cache.plan_kernel(8, 1, max_q=1, max_kv=10) == "kv_attention_team_kernel<1 CTA>"
    assert cache.status() == 0
