"""Plain references in 64 bits for the 8-bit cache and the shared pages, written
from the definitions in include/rra_serve.h."""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------- the 8-bit cache --
def e4m3(y):
    """Bytes of y (float64) rounded to the nearest e4m3, ties to even, saturating."""
    y = np.asarray(y, np.float64)
    m = np.minimum(np.abs(y), 448.0)
    e = np.maximum(np.frexp(m)[1] - 1, -6)  # m = 1.x * 2^e, or below 2^-6
    units = np.rint(np.ldexp(m, 3 - e)).astype(np.int64)  # of 2^(e - 3); 16 carries into the exponent
    return np.where(np.signbit(y), 128, 0).astype(np.int64) | np.where(units == 0, 0, (e + 6) * 8 + units)


def values(codes):
    c = np.asarray(codes, np.int64)
    mag, ex = c & 7, c >> 3 & 15
    v = np.where(ex == 0, mag * 2.0 ** -9, np.ldexp(8.0 + mag, ex - 10))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def at(d):
    """[16, d]: byte of each row and channel in a block's codes."""
    r, c = np.arange(16)[:, None], np.arange(d)[None]
    line, piece = r * d // 128, (r * d % 128 + c) // 16
    return line * 128 + (piece ^ (r & 7 if d == 128 else r & 6)) * 16 + c % 16


def exponent(x):
    """Smallest e in [-32, 32] with max |x| <= 448 * 2^e over what is finite."""
    a = np.abs(np.asarray(x, np.float64))
    most = a[np.isfinite(a)].max(initial=0.0)
    e = -32
    while e < 32 and most > 448.0 * 2.0 ** e:
        e += 1
    return e


def append8(pages, ps, hk, d, k, v, slots):
    """pages: uint8 [num_pages, bytes], changed in place."""
    blocks = pages.reshape(pages.shape[0], hk, ps // 16, 32 * d + 16)
    place, room = at(d), pages.shape[0] * ps
    good = [i for i, s in enumerate(slots) if 0 <= s < room]  # the others are skipped
    k, v, slots = k[good], v[good], [slots[i] for i in good]
    t = 0
    while t < len(slots):
        end = t
        while end < len(slots) and slots[end] // 16 == slots[t] // 16:
            end += 1
        page, i = divmod(int(slots[t]), ps)
        for h in range(hk):
            b = blocks[page, h, i // 16]
            for n, x in enumerate((k, v)):
                part = x[t:end, h].astype(np.float64)
                part = np.where(np.isnan(part), 0.0, part)
                e = exponent(part)
                old = min(max(int(b[32 * d + n:32 * d + n + 1].view(np.int8)[0]), -32), 32)
                codes = b[n * 16 * d:(n + 1) * 16 * d]
                if not any(s % 16 == 0 for s in slots[t:end]):
                    e = max(e, old)
                    if e > old:
                        new = e4m3(np.nan_to_num(values(codes)) * 2.0 ** (old - e))
                        codes[:] = np.where(np.isnan(values(codes)), codes, new)
                for j, s in enumerate(slots[t:end]):
                    codes[place[s % 16]] = e4m3(part[j] * 2.0 ** -e)
                b[32 * d + n] = np.int8(e).view(np.uint8)
        t = end


def read8(pages, ps, hk, d, slots):
    """K and V float64 [len(slots), hk, d]; 0 for slots outside."""
    blocks = pages.reshape(pages.shape[0], hk, ps // 16, 32 * d + 16)
    place = at(d)
    out = np.zeros((2, len(slots), hk, d))
    for t, s in enumerate(slots):
        if 0 <= s < pages.shape[0] * ps:
            page, i = divmod(int(s), ps)
            b = blocks[page, :, i // 16]
            for n in range(2):
                e = np.clip(b[:, 32 * d + n].astype(np.uint8).view(np.int8).astype(np.int64), -32, 32)
                out[n, t] = values(b[:, n * 16 * d + place[i % 16]]) * 2.0 ** e[:, None]
    return out


# ---------------------------------------------------------- shared pages --
def held(n, ps, width):
    return min(-(-max(int(n), 0) // ps), width)


def fork(seq, source, target, table, free, count, shared, ps):
    """table and shared are changed in place; returns kv_len, copy_from, copy_to, free_left, pages_short."""
    seq, pool, width = [int(x) for x in seq], len(free), table.shape[1]
    kv, top, short, frm, to = list(seq), count, 0, [], []
    rows = table.copy()
    for s, t in zip(source, target):
        frm.append(-1)
        to.append(-1)
        if not (0 <= s < len(seq) and 0 <= t < len(seq)):
            continue
        n = max(seq[s], 0)
        full = min(n // ps, width)
        for i in range(full):
            table[t, i] = rows[s, i]
            if 0 <= rows[s, i] < pool:
                shared[rows[s, i]] += 1
        if full < width and n > full * ps:
            page = rows[s, full]
            if 0 <= page < pool:
                fresh = -1
                if top > 0:
                    top -= 1
                    fresh = free[top]
                else:
                    short += 1
                if 0 <= fresh < pool:
                    frm[-1], to[-1] = page, fresh
                else:
                    fresh = -1
                table[t, full] = fresh
            else:
                table[t, full] = page
        kv[t] = n
    return kv, frm, to, top, short


def release(seq, new, table, free, count, shared, ps):
    """free and shared are changed in place; returns kv_len, free_left."""
    pool, width = len(free), table.shape[1]
    holders, drops = shared + 1, np.zeros(pool, np.int64)
    for b in range(len(seq)):
        if new[b] < 0:
            for i in range(held(seq[b], ps, width)):
                if 0 <= table[b, i] < pool:
                    drops[table[b, i]] += 1
    for p in range(pool):
        if drops[p] >= holders[p]:
            shared[p] = 0
            if count < pool:
                free[count] = p
                count += 1
        else:
            shared[p] -= drops[p]
    return [0 if n < 0 else int(s) for s, n in zip(seq, new)], count


def compact(seq, table, free, count, shared, ps, most):
    """Returns table, free, free_left, shared, moved, the moves."""
    pool, width = len(free), table.shape[1]
    is_free = np.zeros(pool, bool)
    for i in range(count):
        if 0 <= free[i] < pool:
            is_free[free[i]] = True
    holes, used = list(np.nonzero(is_free)[0]), list(np.nonzero(~is_free)[0][::-1])
    moves = [(int(s), int(h)) for s, h in zip(used, holes) if s > h][:most]
    moved = np.where(is_free, -1, np.arange(pool))
    shared, table, free = shared.copy(), table.copy(), free.copy()
    for s, h in moves:
        moved[s] = h
        shared[h], shared[s] = shared[s], 0
        is_free[s], is_free[h] = True, False
    for b in range(len(seq)):
        for i in range(held(seq[b], ps, width)):
            if 0 <= table[b, i] < pool:
                table[b, i] = moved[table[b, i]]
    now = np.nonzero(is_free)[0][::-1]
    free[:len(now)] = now
    return table, free, len(now), shared, moved, moves
