"""Plain references in 64 bits for the decode-step operators, and the layout of
the 4-bit cache, written from the definitions in include/rra_serve.h."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def byte_and_shift(d):
    """Byte of a row of codes, and bit of the nibble in it, of every channel."""
    ch = np.arange(d)
    j, c, e = ch // 32, ch % 32 // 4, ch % 4
    return (c * (d // 32) + j) * 2 + e // 2, 4 * (e % 2)


def quantise(x):
    """codes uint8 [..., d] and scales float16 [..., d/32] of x (float32), as the write is defined."""
    x = np.where(np.isnan(x), np.float32(0), x).astype(np.float32)
    g = x.reshape(x.shape[:-1] + (-1, 32))
    with np.errstate(over="ignore", invalid="ignore"):
        s = np.clip(np.abs(g).max(-1) * np.float32(1.0 / 6.0), np.float32(2.0 ** -14), np.float32(2048)).astype(np.float16)
        y = np.abs(g / s.astype(np.float32)[..., None]).astype(np.float64)
    y = np.minimum(y, 6.0)
    high = np.clip(np.searchsorted(E2M1, y), 1, 7)
    low = high - 1
    down, up = y - E2M1[low], E2M1[high] - y
    code = np.where((down < up) | ((down == up) & (low % 2 == 0)), low, high)
    code = code | (np.signbit(g).astype(np.int64) << 3)
    return code.reshape(x.shape).astype(np.uint8), s


def dequantise(codes, scales):
    v = np.where(codes >= 8, -1.0, 1.0) * E2M1[codes & 7]
    return v * np.repeat(scales.astype(np.float64), 32, -1)


def write_pages(pages, ps, hk, d, k, v, slots):
    """pages: uint8 [num_pages, bytes] changed in place."""
    blocks = pages.reshape(-1, hk, ps // 16, 18 * d)
    at, shift = byte_and_shift(d)
    n = pages.shape[0] * ps
    for x, c, s in ((k, 0, 16 * d), (v, 8 * d, 17 * d)):
        codes, scales = quantise(x)
        row = np.zeros(codes.shape[:-1] + (d // 2,), dtype=np.uint8)
        for ch in range(d):
            row[..., at[ch]] |= codes[..., ch] << np.uint8(shift[ch])
        raw = np.ascontiguousarray(scales).view(np.uint8)
        for t, slot in enumerate(slots):
            if 0 <= slot < n:
                page, i = divmod(int(slot), ps)
                b = blocks[page, :, i // 16]
                b[:, c + i % 16 * (d // 2):c + (i % 16 + 1) * (d // 2)] = row[t]
                b[:, s + i % 16 * (d // 16):s + (i % 16 + 1) * (d // 16)] = raw[t]


def read_pages(pages, ps, hk, d, slots):
    """K and V float64 [len(slots), hk, d]; 0 for slots outside."""
    blocks = pages.reshape(-1, hk, ps // 16, 18 * d)
    at, shift = byte_and_shift(d)
    out = np.zeros((2, len(slots), hk, d))
    for t, slot in enumerate(slots):
        if 0 <= slot < pages.shape[0] * ps:
            page, i = divmod(int(slot), ps)
            b = blocks[page, :, i // 16]
            for n, (c, s) in enumerate(((0, 16 * d), (8 * d, 17 * d))):
                codes = b[:, c + i % 16 * (d // 2) + at] >> shift & 15
                scales = np.ascontiguousarray(b[:, s + i % 16 * (d // 16):s + (i % 16 + 1) * (d // 16)]).view(np.float16)
                out[n, t] = dequantise(codes, scales)
    return out


def attention(q, keys, values, kv, scale, causal, window, seen=None):
    """q [n, hq, d], keys and values [kv, hk, d], all float64.  Returns out, lse,
    mean |v| under the weights, and the largest sum of |q_i k_i| * |scale|."""
    n, hq, d = q.shape
    hk = keys.shape[1]
    out, lse = np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
    mean, dots = np.zeros((n, hq, d)), np.zeros((n, hq))
    for i in range(n):
        pos = kv - n + i
        see = np.ones(kv, dtype=bool) if seen is None else seen.copy()
        key = np.arange(kv)
        if causal:
            see &= key <= pos
        if window:
            see &= key > pos - window
        if not see.any():
            continue
        for h in range(hq):
            k, v = keys[see, h * hk // hq], values[see, h * hk // hq]
            s = k @ q[i, h] * scale
            m = s.max()
            p = np.exp(s - m)
            out[i, h], lse[i, h] = p @ v / p.sum(), m + np.log(p.sum())
            mean[i, h], dots[i, h] = p @ np.abs(v) / p.sum(), (np.abs(k) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, mean, dots


def norm_rope(x, w, cos, sin, pos, eps, interleaved):
    """x [t, heads, d] float64; w [d] or None; cos, sin [p, rot/2].  Returns the
    result and the size of what was added for each channel."""
    y = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    size = np.abs(y)
    if cos is None or cos.shape[1] == 0:
        return y, size
    half = cos.shape[1]
    y, size = y.copy(), size.copy()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    good = (pos >= 0) & (pos < cos.shape[0])
    p = np.where(good, pos, 0)
    c = np.where(good[:, None], cos[p], np.nan)[:, None]
    s = np.where(good[:, None], sin[p], np.nan)[:, None]
    u, v = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    size[..., a] = size[..., b] = np.abs(u) + np.abs(v)
    return y, size


def slot_map(seq, new, table, free, count, ps, tokens):
    """One bookkeeping step in plain loops; table and free are changed in place."""
    pool, width = len(free), table.shape[1]
    top, up = count, lambda x: -(-x // ps)
    for b in range(len(seq)):
        if new[b] < 0:
            for i in range(min(up(max(seq[b], 0)), width)):
                if 0 <= table[b, i] < pool and top < pool:
                    free[top] = table[b, i]
                    top += 1
    short, slots, positions, kv, cu = 0, [], [], [], [0]
    for b in range(len(seq)):
        held = 0 if new[b] < 0 else max(int(seq[b]), 0)
        add = max(int(new[b]), 0)
        for i in range(up(held), up(held + add)):
            if i >= width:
                short += 1
            elif top > 0:
                top -= 1
                table[b, i] = free[top]
            else:
                table[b, i] = -1
                short += 1
        for i in range(held, held + add):
            page = table[b, i // ps] if i // ps < width else -1
            slots.append(int(page) * ps + i % ps if page >= 0 else -1)
            positions.append(i)
        kv.append(held + add)
        cu.append(cu[-1] + add)
    pad = max(0, tokens - len(slots))
    return (kv, cu, (slots + [-1] * pad)[:tokens], (positions + [0] * pad)[:tokens], top, short)


def leave_zeros():
    """Overwrites what the allocator keeps with zeros, for tests that come later.  These tests fill tables with -1 and pages
    with NaN patterns; the sentinel AllReduces take a buffer of all-ones for data that has not arrived, and tests enqueue them
    on buffers straight from the allocator."""
    import gc

    import torch

    gc.collect()
    torch.cuda.synchronize()
    for size in (1 << 20, 2 << 20):  # its pools of small and of large blocks
        before, kept = torch.cuda.memory_reserved(), []
        while torch.cuda.memory_reserved() == before:
            kept.append(torch.zeros(size, dtype=torch.uint8, device="cuda"))
        del kept
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
