"""Pages that requests share, on a GPU, against plain loops."""
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


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def zeros(n):
    return torch.full((n,), -77, dtype=torch.int32, device="cuda")


def eq(got, want):
    got = got.cpu().numpy()
    assert np.array_equal(got, np.asarray(want)), (got[:20], np.asarray(want)[:20])


def state(rng, lengths, ps, pool, rows, width=None):
    """Tables of requests with these lengths (and empty rows), the stack, its count, counts of holders."""
    held = [-(-max(n, 0) // ps) for n in lengths]
    width = max(held + [1]) + 1 if width is None else width
    order = rng.permutation(pool)
    table = np.full((rows, width), -1, np.int32)
    used = 0
    for b, h in enumerate(held):
        n = min(h, width)
        table[b, :n] = order[used:used + n]
        used += n
    free = np.full(pool, -5, np.int32)
    free[:pool - used] = order[used:]
    seq = np.array(list(lengths) + [0] * (rows - len(lengths)), np.int32)
    return seq, table, free, pool - used, np.zeros(pool, np.int32)


FORKS = {
    # name: lengths, page_tokens, pool, rows, sources, targets, free pages left (None: all)
    "one into one": ([100], 16, 40, 2, [0], [1], None),
    "whole pages only": ([64], 16, 40, 3, [0, 0], [1, 2], None),
    "less than a page": ([3], 16, 40, 4, [0, 0, 0], [1, 2, 3], None),
    "nothing": ([0, 5], 16, 40, 4, [0, 0], [2, 3], None),
    "none": ([5], 16, 40, 4, [], [], None),
    "a negative length": ([-4, 5], 16, 40, 4, [0, 1], [2, 3], None),
    "rows that are not there": ([20, 5], 16, 40, 4, [0, 7, -1, 1, 1], [9, 2, 2, -3, 3], None),
    "pages run short": ([20, 5, 33], 16, 40, 10, [0, 1, 2, 0, 1], [5, 6, 7, 8, 9], 2),
    "no pages left": ([20, 5], 16, 40, 4, [0, 1], [2, 3], 0),
    "many": (list(range(1, 400, 7)), 16, 4000, 500, [i % 58 for i in range(300)], list(range(60, 360)), None),
    "long rows": ([16 * 700 + 3, 16 * 300], 16, 1400, 40, [0] * 20 + [1] * 10, list(range(2, 32)), None),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", sorted(FORKS))
def test_fork(serve, case, in_place):
    lengths, ps, pool, rows, source, target, left = FORKS[case]
    seq, table, free, count, shared = state(np.random.default_rng(1), lengths, ps, pool, rows)
    count = count if left is None else left
    shared[::3] = 2
    d_seq, d_table, d_free, d_count, d_shared = (dev(x) for x in (seq, table, free, [count], shared))
    kv, out, fl = (d_seq, d_shared, d_count) if in_place else (zeros(rows), zeros(pool), zeros(1))
    frm, to, short = zeros(len(source)), zeros(len(source)), zeros(1)
    serve.pages_fork(d_seq, dev(source), dev(target), d_table, d_free, d_count, d_shared, ps, kv_len=kv, shared_out=out,
                     copy_from=frm, copy_to=to, free_left=fl, pages_short=short)
    want = more.fork(seq, source, target, table, free, count, shared, ps)
    eq(kv, want[0])
    eq(frm, want[1])
    eq(to, want[2])
    eq(fl, [want[3]])
    eq(short, [want[4]])
    eq(d_table, table)
    eq(out, shared)
    eq(d_free, free)


def test_fork_with_a_corrupt_table_and_stack(serve):
    """Numbers that are no pages are copied or left out; nothing outside the buffers is touched."""
    ps, pool = 16, 30
    seq, table, free, count, shared = state(np.random.default_rng(2), [40, 40, 50], ps, pool, 9)
    table[0, 1], table[1, 2], table[2, 3] = 10 ** 9, -1, 2 ** 31 - 1
    free[count - 1], free[count - 2] = 10 ** 8, -3
    source, target = [0, 1, 2, 0, 0], [4, 5, 6, 7, 8]
    d = [dev(x) for x in (seq, table, free, [count], shared)]
    kv, out, fl, frm, to, short = zeros(9), zeros(pool), zeros(1), zeros(5), zeros(5), zeros(1)
    serve.pages_fork(d[0], dev(source), dev(target), d[1], d[2], d[3], d[4], ps, kv_len=kv, shared_out=out, copy_from=frm,
                     copy_to=to, free_left=fl, pages_short=short)
    want = more.fork(seq, source, target, table, free, count, shared, ps)
    for got, w in zip((kv, frm, to), want):
        eq(got, w)
    eq(d[1], table)
    eq(out, shared)


RELEASES = {
    # name: lengths, page_tokens, pool, new_len, rows (b, a): b begins with a's first whole pages
    "none ends": ([40, 9], 16, 20, [1, 0], []),
    "one": ([40, 9, 70], 16, 20, [1, -1, 3], []),
    "all": ([40, 9, 70], 16, 20, [-1, -5, -1], []),
    "a holder of two": ([40, 70, 9], 16, 30, [-1, 1, 1], [(1, 0)]),
    "the last holders": ([40, 70, 99], 16, 30, [-1, -1, 2], [(1, 0), (2, 0)]),
    "every holder": ([40, 70, 99], 16, 30, [-1, -1, -1], [(1, 0), (2, 0)]),
    "no requests": ([], 16, 30, [], []),
    "many": ([(37 * i) % 500 for i in range(700)], 16, 13001, [-1 if i % 3 else 1 for i in range(700)],
             [(i, i - 1) for i in range(1, 700, 2)]),
    "a large pool": ([100, 5000], 16, 300000, [-1, -1], []),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", sorted(RELEASES))
def test_release(serve, case, in_place):
    lengths, ps, pool, new, common = RELEASES[case]
    rows = len(lengths)
    seq, table, free, count, shared = state(np.random.default_rng(3), lengths, ps, pool, rows, 400)
    for b, a in common:
        for i in range(min(lengths[a], lengths[b]) // ps):
            free[count] = table[b, i]
            count += 1
            table[b, i] = table[a, i]
            shared[table[a, i]] += 1
    d_seq, d_new, d_table, d_free, d_count, d_shared = (dev(x) for x in (seq, new, table, free, [count], shared))
    kv, out, fl = (d_seq, d_shared, d_count) if in_place else (zeros(rows), zeros(pool), zeros(1))
    serve.pages_release(d_seq, d_new, d_table, d_free, d_count, d_shared, ps, kv_len=kv, shared_out=out, free_left=fl)
    want = more.release(seq, new, table, free, count, shared, ps)
    eq(kv, want[0])
    eq(fl, [want[1]])
    eq(out, shared)
    eq(d_free, free)
    eq(d_table, table)


def test_release_with_a_corrupt_table(serve):
    """A page listed too often goes back once; numbers that are no pages, and what would not fit the stack, are left out."""
    ps, pool = 16, 12
    table = np.array([[3, 3, 3, 99, -1, 7], [3, 8, 1, 0, 0, 0]], np.int32)
    seq, new, free = [96, 40], [-1, -1], np.arange(pool, dtype=np.int32)
    for count in (2, 10, 12, 50, -3):
        shared, f = np.zeros(pool, np.int32), free.copy()
        d = [dev(x) for x in (seq, new, table, f, [count], shared)]
        kv, fl = zeros(2), zeros(1)
        serve.pages_release(*d, ps, kv_len=kv, shared_out=d[5], free_left=fl)
        want = more.release(seq, new, table, f, min(max(count, 0), pool), shared, ps)
        eq(kv, want[0])
        eq(fl, [want[1]])
        eq(d[5], shared)
        eq(d[3], f)


COMPACTS = {
    # name: lengths, page_tokens, pool, moves
    "nothing free": ([64, 48], 16, 7, 4),
    "all free": ([0, 0], 16, 7, 4),
    "few": ([40, 9, 70], 16, 20, 20),
    "a budget": ([40, 9, 70, 300], 16, 90, 5),
    "no moves": ([40, 9, 70, 300], 16, 90, 0),
    "no pages": ([0], 16, 0, 3),
    "odd": ([16 * 50 + 1, 7], 16, 101, 77),
    "many": ([(37 * i) % 500 for i in range(700)], 16, 20011, 10000),
    "many, a budget": ([(37 * i) % 500 for i in range(700)], 16, 20011, 777),
    "a large pool": ([1000, 5000], 16, 300000, 1000),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", sorted(COMPACTS))
def test_compact(serve, case, in_place):
    lengths, ps, pool, most = COMPACTS[case]
    rng = np.random.default_rng(4)
    seq, table, free, count, shared = state(rng, lengths, ps, pool, len(lengths))
    used = np.ones(pool, bool)
    used[free[:count]] = False
    shared[used] = rng.integers(0, 5, used.sum())
    if lengths[0] > 32:
        table[-1, -1] = table[0, 0]  # an entry that the request does not hold
    d_seq, d_table, d_free, d_count, d_shared = (dev(x) for x in (seq, table, free, [count], shared))
    wide = torch.full((len(lengths), table.shape[1] + 3), -77, dtype=torch.int32, device="cuda")
    t_out, f_out, fl, s_out = (d_table, d_free, d_count, d_shared) if in_place else \
        (wide[:, 1:-2], d_free.clone(), zeros(1), zeros(pool))
    moved, frm, to, n = zeros(pool), zeros(most), zeros(most), zeros(1)
    serve.pages_compact(d_seq, d_table, d_free, d_count, d_shared, ps, table_out=t_out, free_out=f_out, shared_out=s_out,
                        free_left=fl, moved=moved, move_from=frm, move_to=to, move_count=n)
    table, free, left, shared, want_moved, moves = more.compact(seq, table, free, count, shared, ps, most)
    eq(n, [len(moves)])
    eq(frm, [s for s, _ in moves] + [-1] * (most - len(moves)))
    eq(to, [h for _, h in moves] + [-1] * (most - len(moves)))
    eq(moved, want_moved)
    eq(fl, [left])
    eq(f_out, free)
    eq(s_out, shared)
    eq(t_out, table)
    if not in_place:
        assert (wide[:, 0] == -77).all() and (wide[:, -2:] == -77).all()
    if most >= pool // 2 and pool:
        assert left == count and (left == 0 or free[left - 1] == pool - left)


def test_compact_with_a_corrupt_stack(serve):
    """Numbers that are no pages, or come twice, count for what they are."""
    ps, pool = 16, 20
    seq, table, free, count, shared = state(np.random.default_rng(5), [100, 40], ps, pool, 2)
    free[1], free[3], free[4] = 99, free[2], -7
    d = [dev(x) for x in (seq, table, free, [count], shared)]
    t_out, f_out, s_out, fl, moved, frm, to, n = dev(table), dev(free), zeros(pool), zeros(1), zeros(pool), zeros(9), zeros(9), zeros(1)
    serve.pages_compact(*d, ps, table_out=t_out, free_out=f_out, shared_out=s_out, free_left=fl, moved=moved, move_from=frm,
                        move_to=to, move_count=n)
    table, free, left, shared, want_moved, moves = more.compact(seq, table, free, count, shared, ps, 9)
    eq(n, [len(moves)])
    eq(moved, want_moved)
    eq(fl, [left])
    eq(f_out, free)
    eq(t_out, table)


@pytest.mark.parametrize("kind", ["KvCache", "KvCache8"])
@pytest.mark.parametrize("d,ps,hk,pool", [(64, 16, 1, 9), (128, 64, 3, 40), (128, 4096, 2, 6)])
def test_copy(serve, kind, d, ps, hk, pool):
    cls = getattr(serve, kind)
    size = serve.kv_page_bytes(ps, hk, d) if kind == "KvCache" else serve.kv8_page_bytes(ps, hk, d)
    a, b = (cls(torch.randint(0, 256, (n, size), dtype=torch.uint8, device="cuda"), ps, hk, d) for n in (pool, pool + 2))
    was_a, was_b = a.pages.clone(), b.pages.clone()
    a.copy(dev([0, -1, 3, 2, 1]), dev([4, 1, -1, pool, pool - 1]))
    want = was_a.clone()
    want[4] = was_a[0]
    want[pool - 1] = was_a[1]
    assert torch.equal(a.pages, want)
    a.copy(dev([0, pool, 2]), dev([pool + 1, 0, 1]), to=b)
    was_b[pool + 1] = want[0]
    was_b[1] = want[2]
    assert torch.equal(b.pages, was_b) and torch.equal(a.pages, want)
    a.copy(dev([]), dev([]))
    other = cls(torch.zeros(2, size * 2, dtype=torch.uint8, device="cuda"), ps, hk * 2, d)
    with pytest.raises(ValueError):
        a.copy(dev([0]), dev([1]), to=other)


def test_bookkeeping_in_a_graph(serve):
    """Fork and release undo each other, whatever the number of replays."""
    ps, pool = 16, 500
    rng = np.random.default_rng(7)
    seq, table, free, count, shared = state(rng, [100, 64, 33], ps, pool, 9)
    d_seq, d_table, d_free, d_count, d_shared = (dev(x) for x in (seq, table, free, [count], shared))
    frm, to, short = zeros(6), zeros(6), zeros(1)
    source, target = dev([0, 0, 1, 1, 2, 2]), dev([3, 4, 5, 6, 7, 8])
    new = dev([1, 1, 1] + [-1] * 6)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        serve.pages_fork(d_seq, source, target, d_table, d_free, d_count, d_shared, ps, kv_len=d_seq, shared_out=d_shared,
                         copy_from=frm, copy_to=to, free_left=d_count, pages_short=short)
        serve.pages_release(d_seq, new, d_table, d_free, d_count, d_shared, ps, kv_len=d_seq, shared_out=d_shared, free_left=d_count)
    for _ in range(5):
        graph.replay()
        eq(d_seq, seq)
        eq(d_count, [count])
        eq(d_shared, shared)
        assert sorted(d_free.tolist()[:count]) == sorted(free[:count])
        assert short.item() == 0 and (to.cpu() >= 0).sum() == 4
