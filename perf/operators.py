"""Cases of the decode-step operators (latency_barrier_free_gb300/serve.py).

Around the AllReduces of a tensor-parallel decode step a serving program has,
for every token: the page bookkeeping of its key/value cache (`slots`), the
norms and the position rotation of queries and keys (`rope`), the write into a
cache held in 4 bits and the read back of what it stands for (`store`), and the
attention over that cache (`attend`).  A case names one of these four and its
sizes.  `run` computes it in plain torch operations in 32 bits, or, with `own`
set, by the package's operators; `exact` computes it in 64 bits.

The 4-bit cache.  A page holds `ps` tokens (a multiple of 16) of every KV head:
bytes [head][block of 16 tokens][18 * d].  A block of 16 tokens is K codes
(16 x d/2), V codes (16 x d/2), K scales (16 x d/32 binary16), V scales.  A
code is e2m1 (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives); 32 neighbouring
channels share a scale; channel 32 j + 4 c + e of a row is in byte
(c * d/32 + j) * 2 + e/2, its low nibble for even e.
"""
import math
import random

import torch

own = False

GROUP = 32  # channels that share a scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SCALE_MIN, SCALE_MAX = 2.0 ** -14, 2048.0


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one decode step of 64 requests, a token each: pure latency
        {"name": "slots, 64 decoding", "op": "slots", "requests": 64, "tokens": 64, "longest": 8192, "ps": 64},
        # continuous batching at the largest: most requests decode, some bring a prompt, some end
        {"name": "slots, 1000 mixed", "op": "slots", "requests": 1000, "tokens": 65536, "longest": 16384, "ps": 16},
        # queries and keys of 4 tokens of the [B, 8192] decode step: 64 heads over 8 KV heads
        {"name": "rope, 4 tokens", "op": "rope", "tokens": 4, "hq": 64, "hk": 8, "d": 128, "rot": 128,
         "pairs": "halves", "dtype": "bf16"},
        # a prompt of the same model, rows of the packed projection (strided)
        {"name": "rope, 8192 tokens", "op": "rope", "tokens": 8192, "hq": 64, "hk": 8, "d": 128, "rot": 128,
         "pairs": "halves", "dtype": "bf16"},
        # binary32, a part of each head rotated, neighbouring channels paired, odd counts
        {"name": "rope, 1021 odd fp32", "op": "rope", "tokens": 1021, "hq": 9, "hk": 3, "d": 64, "rot": 48,
         "pairs": "neighbours", "dtype": "fp32"},
        # the cache write of a decode step, and what it stands for
        {"name": "store, 16 tokens", "op": "store", "tokens": 16, "hk": 8, "d": 128, "ps": 64, "dtype": "bf16"},
        # the cache write of a long prompt
        {"name": "store, 16384 tokens", "op": "store", "tokens": 16384, "hk": 8, "d": 128, "ps": 64, "dtype": "bf16"},
        # one request on one tensor-parallel rank (8 heads, 1 KV head): latency
        {"name": "attend, 1 x 2000", "op": "attend", "requests": 1, "queries": 1, "longest": 2000, "hq": 8, "hk": 1,
         "d": 128, "ps": 64, "causal": True, "window": 0},
        # a decode batch of 64 ragged requests, all heads, some padding
        {"name": "attend, 64 ragged", "op": "attend", "requests": 64, "queries": 1, "longest": 16384, "hq": 64,
         "hk": 8, "d": 128, "ps": 64, "causal": True, "window": 0},
        # one long context, all heads
        {"name": "attend, 1 x 131071", "op": "attend", "requests": 1, "queries": 1, "longest": 131071, "hq": 64,
         "hk": 8, "d": 128, "ps": 64, "causal": True, "window": 0},
        # a few drafted tokens to verify, odd groups of 7 heads, small heads, sliding window
        {"name": "attend, verify 5", "op": "attend", "requests": 24, "queries": 5, "longest": 4099, "hq": 14, "hk": 2,
         "d": 64, "ps": 16, "causal": True, "window": 1000},
        # prompts in chunks on top of what the cache already holds
        {"name": "attend, prompt chunks", "op": "attend", "requests": 3, "queries": 1024, "longest": 8192, "hq": 64,
         "hk": 8, "d": 128, "ps": 64, "causal": True, "window": 0},
    ]


def _log(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["slots", "rope", "rope", "store", "attend", "attend", "attend"])
    d, ps = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    if op == "slots":
        requests = _log(rng, 1, 1000)
        return {"op": op, "requests": requests, "tokens": requests + _log(rng, 1, 65536), "ps": ps,
                "longest": _log(rng, 64, 16384)}
    if op == "rope":
        hk = _log(rng, 1, 8)
        return {"op": op, "tokens": _log(rng, 1, 8192), "hq": hk * rng.randint(1, 8), "hk": hk, "d": d,
                "rot": rng.choice([d, d, d // 2, d // 4 * 3]), "pairs": rng.choice(["halves", "neighbours"]),
                "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "store":
        return {"op": op, "tokens": _log(rng, 1, 16384), "hk": _log(rng, 1, 8), "d": d, "ps": ps,
                "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    hk, group = _log(rng, 1, 8), rng.choice([1, 2, 4, 5, 7, 8, 8, 16])
    queries = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 1024)])
    most = 2 ** 20 if queries == 1 else 2 ** 18 if queries <= 8 else 24576  # keys of all requests together
    longest = _log(rng, max(queries, 16), 131071 if queries <= 8 else 8192)
    return {"op": op, "requests": _log(rng, 1, max(1, min(64, most // longest))), "queries": queries,
            "longest": longest, "hq": hk * min(group, 64 // hk), "hk": hk, "d": d, "ps": ps,
            "causal": rng.random() < 0.9, "window": rng.choice([0, 0, 0, _log(rng, 16, 4096)])}


def _lengths(case):
    """Query and key counts of each request; they go by the case alone, so that work() knows them."""
    rng = random.Random("%(requests)d %(queries)d %(longest)d" % case)
    n = case["requests"]
    new = [case["queries"]] + [_log(rng, 1, case["queries"]) for _ in range(n - 1)]
    kv = [case["longest"]] + [max(q, _log(rng, 16, case["longest"])) for q in new[1:]]
    if n >= 16:
        kv[-1], kv[-2] = 0, 1  # a padding request, whose rows see no key, and one whose first token this is
        new[-2] = 1
    return new, kv


def _step(case):
    """Tokens held and tokens to add (negative: the request ends) of each request of a page bookkeeping step."""
    rng = random.Random("%(requests)d %(tokens)d %(longest)d %(ps)d" % case)
    n, spare = case["requests"], case["tokens"] - case["requests"]
    held = [_log(rng, 1, case["longest"]) for _ in range(n)]
    new = [1] * n
    for b in range(n):
        if n >= 16 and b % 16 == 7:
            new[b] = -1
        elif spare > 0 and (n < 16 or b % 16 == 3):  # a prompt: nothing held yet
            held[b], more = 0, min(spare, _log(rng, 16, case["longest"]))
            new[b], spare = more, spare - more
    return held, new


def work(case):
    if case["op"] == "slots":
        held, new = _step(case)
        ps, up = case["ps"], lambda x: -(-x // case["ps"])
        moved = sum(up(h) if q < 0 else up(h + q) - up(h) for h, q in zip(held, new))
        return {"bytes": 16 * len(held) + 12 * case["tokens"] + 8 * moved, "flops": 0}
    size = {"bf16": 2, "fp32": 4}.get(case.get("dtype"), 2)
    d = case["d"]
    if case["op"] == "rope":
        values = case["tokens"] * (case["hq"] + case["hk"]) * d
        return {"bytes": 2 * size * values + case["tokens"] * (4 + 4 * case["rot"]), "flops": 8 * values}
    if case["op"] == "store":  # values in, codes and scales out and in, values out
        values = 2 * case["tokens"] * case["hk"] * d
        return {"bytes": values * 2 * size + 2 * values * 9 // 16 + 8 * case["tokens"], "flops": 6 * values}
    new, kv = _lengths(case)
    pairs = keys = 0
    for n, length in zip(new, kv):
        first = length
        for i in range(n):
            end = min(length, max(0, length - n + i + 1)) if case["causal"] else length
            begin = max(0, length - n + i + 1 - case["window"]) if case["window"] else 0
            pairs += max(0, end - begin)
            first = min(first, begin)
        keys += length - first
    return {"bytes": keys * case["hk"] * d * 9 // 8 + 4 * sum(new) * case["hq"] * (d + 1),
            "flops": 4 * pairs * case["hq"] * d}


# ----------------------------------------------------- the 4-bit cache, plain --
def _const(values, device, dtype=torch.float32):
    return torch.tensor(values, dtype=dtype, device=device)


def _quantise(x):
    """(codes 0..15, scales binary16) of the rows x [..., d]: the scale is the group's largest magnitude / 6."""
    x = torch.nan_to_num(x.float(), nan=0.0, posinf=math.inf, neginf=-math.inf)
    g = x.unflatten(-1, (-1, GROUP))
    s = (g.abs().amax(-1) * (1.0 / 6.0)).clamp(SCALE_MIN, SCALE_MAX).to(torch.float16)
    y = (g / s.float()[..., None]).abs()
    m = torch.zeros_like(y, dtype=torch.uint8)
    for k in range(7):  # midpoints of neighbouring codes; a tie goes to the even code
        mid = (E2M1[k] + E2M1[k + 1]) / 2
        m += (y > mid) if k % 2 == 0 else (y >= mid)
    return ((m | (torch.signbit(g).to(torch.uint8) << 3)).flatten(-2), s)


def _pack(codes):
    """codes [..., d] -> bytes [..., d/2] in the cache's channel order."""
    c = codes.unflatten(-1, (-1, 8, 4)).transpose(-3, -2).flatten(-3)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _values(codes, scales, lut):
    """bytes [..., d/2], scales [..., d/32] -> values [..., d] in 32 bits."""
    j = scales.shape[-1]
    v = lut[codes.int()].flatten(-2).unflatten(-1, (8, j, 4)).transpose(-3, -2).flatten(-2)
    return (v * scales.float()[..., None]).flatten(-2)


def _pairs(device):
    """The two values of each byte."""
    table = E2M1 + tuple(-v for v in E2M1)
    return _const([[table[b & 15], table[b >> 4]] for b in range(256)], device)


def _parts(block, d):
    """K codes, V codes, K scales, V scales of blocks [..., 18 d]."""
    c, s = 8 * d, d
    k, v = block[..., :c].unflatten(-1, (16, d // 2)), block[..., c:2 * c].unflatten(-1, (16, d // 2))
    ks = block[..., 2 * c:2 * c + s].contiguous().view(torch.float16).unflatten(-1, (16, d // GROUP))
    vs = block[..., 2 * c + s:].contiguous().view(torch.float16).unflatten(-1, (16, d // GROUP))
    return k, v, ks, vs


def _fill(pages, case, gen):
    """Keys and values of normal size, quantised into every page; every head has a size of its own, as real ones do."""
    d, hk, ps = case["d"], case["hk"], case["ps"]
    blocks = pages.view(-1, hk, ps // 16, 18 * d)
    step = max(1, (1 << 26) // (hk * ps * d))
    for at in range(0, blocks.shape[0], step):
        part = blocks[at:at + step]
        for n, (c, s) in enumerate(((0, 16 * d), (8 * d, 17 * d))):
            x = torch.randn(part.shape[:3] + (16, d), generator=gen, device=pages.device)
            x *= torch.linspace(0.5, 2.0, hk, device=pages.device)[:, None, None, None] * (1.0 if n == 0 else 0.3)
            codes, scales = _quantise(x)
            part[..., c:c + 8 * d] = _pack(codes).flatten(-2)
            part[..., s:s + d] = scales.flatten(-2).contiguous().view(torch.uint8)


def _page_bytes(case):
    return case["hk"] * case["ps"] // 16 * 18 * case["d"]


# ---------------------------------------------------------------- prepare --
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case, "op": case["op"]}
    _PREPARE[case["op"]](st, case, gen)
    if own and case["op"] in ("store", "attend"):
        from latency_barrier_free_gb300 import serve

        st["cache"] = serve.KvCache(st["pages"], case["ps"], case["hk"], case["d"])
    return st


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _prepare_slots(st, case, gen):
    held, new = _step(case)
    ps, n = case["ps"], case["requests"]
    width = max(-(-max(h, h + q) // ps) for h, q in zip(held, new)) + 1
    pages_held = [-(-h // ps) for h in held]
    pool = sum(-(-max(h, h + q) // ps) for h, q in zip(held, new)) + 64
    order = torch.randperm(pool, generator=gen, device="cuda").int()  # pages are handed out in the order of past traffic
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    inside = torch.arange(width, device="cuda")[None] < torch.tensor(pages_held, device="cuda")[:, None]
    used = sum(pages_held)
    table[inside] = order[:used]
    free = torch.zeros(pool, dtype=torch.int32, device="cuda")
    free[:pool - used] = order[used:]
    st.update(seq_len=_ints(held), new_len=_ints(new), table=table, free=free, free_count=_ints([pool - used]))
    st["out"] = {"kv_len": _ints([0] * n), "cu_new": _ints([0] * (n + 1)), "free_left": _ints([0]),
                 "pages_short": _ints([0]), "positions": _ints([0] * case["tokens"]),
                 "slots": torch.zeros(case["tokens"], dtype=torch.int64, device="cuda")}


def _prepare_rope(st, case, gen):
    t, hq, hk, d, rot = (case[k] for k in ("tokens", "hq", "hk", "d", "rot"))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    qkv = torch.randn(t, hq + 2 * hk, d, generator=gen, device="cuda").to(dt)  # the packed projection
    most = max(2 * t, 8192)
    angle = torch.arange(most, dtype=torch.float64)[:, None] * 500000.0 ** (-torch.arange(0, rot, 2) / rot).double()
    st.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], cos=angle.cos().float().cuda(), sin=angle.sin().float().cuda(),
              wq=(1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dt),
              wk=(1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dt),
              positions=torch.randint(0, most, (t,), generator=gen, device="cuda").int(),
              q_out=torch.empty(t, hq, d, dtype=dt, device="cuda"), k_out=torch.empty(t, hk, d, dtype=dt, device="cuda"))


def _prepare_store(st, case, gen):
    t, hk, d, ps = (case[k] for k in ("tokens", "hk", "d", "ps"))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    pool = -(-t // ps) + 8
    size = torch.linspace(0.5, 2.0, hk, device="cuda")[:, None]
    order = torch.randperm(pool, generator=gen, device="cuda")
    at = torch.arange(t, device="cuda")
    st.update(k=(torch.randn(t, hk, d, generator=gen, device="cuda") * size).to(dt),
              v=(0.3 * torch.randn(t, hk, d, generator=gen, device="cuda") * size).to(dt),
              slots=order[at // ps] * ps + at % ps, pages=torch.zeros(pool, _page_bytes(case), dtype=torch.uint8, device="cuda"),
              k_out=torch.empty(t, hk, d, dtype=dt, device="cuda"), v_out=torch.empty(t, hk, d, dtype=dt, device="cuda"))


def _prepare_attend(st, case, gen):
    new, kv = _lengths(case)
    ps, t = case["ps"], sum(new)
    held = [-(-n // ps) for n in kv]
    pool, width = sum(held) + 4, max(held)
    order = torch.randperm(pool, generator=gen, device="cuda").int()
    table = torch.full((len(new), width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None] < torch.tensor(held, device="cuda")[:, None]] = order[:sum(held)]
    pages = torch.zeros(pool, _page_bytes(case), dtype=torch.uint8, device="cuda")
    _fill(pages, case, gen)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = torch.randn(t, case["hq"], case["d"], generator=gen, device="cuda").bfloat16()
    st.update(q=q, cu_q=_ints(cu), kv_len=_ints(kv), table=table, pages=pages, out=torch.empty_like(q),
              lse=torch.empty(t, case["hq"], device="cuda"))


_PREPARE = {"slots": _prepare_slots, "rope": _prepare_rope, "store": _prepare_store, "attend": _prepare_attend}


# -------------------------------------------------------------------- run --
def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state, state["case"])


def _own_slots(st, case):
    from latency_barrier_free_gb300 import serve

    o = st["out"]
    serve.slot_map(st["seq_len"], st["new_len"], st["table"], st["free"], st["free_count"], case["ps"],
                   kv_len=o["kv_len"], cu_new=o["cu_new"], slots=o["slots"], positions=o["positions"],
                   free_left=o["free_left"], pages_short=o["pages_short"])
    return dict(o, table=st["table"], free=st["free"])


def _own_rope(st, case):
    from latency_barrier_free_gb300 import serve

    serve.qk_norm_rope(st["q"], st["k"], st["wq"], st["wk"], st["cos"], st["sin"], st["positions"], st["q_out"],
                       st["k_out"], eps=1e-6, interleaved=case["pairs"] == "neighbours")
    return {"q": st["q_out"], "k": st["k_out"]}


def _own_store(st, case):
    st["cache"].append(st["k"], st["v"], st["slots"])
    st["cache"].read(st["slots"], st["k_out"], st["v_out"])
    return {"k": st["k_out"], "v": st["v_out"]}


def _own_attend(st, case):
    st["cache"].attention(st["q"], st["out"], st["cu_q"], st["kv_len"], st["table"], max_q=case["queries"],
                          max_kv=case["longest"], causal=case["causal"], window=case["window"], lse=st["lse"])
    return {"out": st["out"], "lse": st["lse"]}


_OWN = {"slots": _own_slots, "rope": _own_rope, "store": _own_store, "attend": _own_attend}


def _plain_slots(st, case):
    ps, table, free = case["ps"], st["table"], st["free"]
    n, width, pool = table.shape[0], table.shape[1], free.numel()
    held, new = st["seq_len"].long().clamp(min=0), st["new_len"].long()
    ends, new = new < 0, new.clamp(min=0)
    col = torch.arange(width, device=table.device)
    # pages of requests that end go on top of the stack, in the order of the requests
    back = ends[:, None] & (col < ((held + ps - 1) // ps)[:, None]) & (table >= 0) & (table < pool)
    place = st["free_count"].long() + back.flatten().cumsum(0).view_as(back) - 1
    spare = torch.cat([free, free.new_zeros(1)])
    spare.scatter_(0, torch.where(back & (place < pool), place, pool).flatten(), table.flatten())
    free.copy_(spare[:pool])
    top = (st["free_count"].long() + back.sum()).clamp(max=pool)
    # new pages come off the top, in the order of the requests
    held = torch.where(ends, 0, held)
    total = held + new
    first, last = (held + ps - 1) // ps, (total + ps - 1) // ps
    fresh = (col >= first[:, None]) & (col < last[:, None])
    i = fresh.flatten().cumsum(0).view_as(fresh) - 1
    page = torch.where(i < top, free[(top - 1 - i).clamp(0, pool - 1)], -1)
    table.copy_(torch.where(fresh, page, table))
    wanted = fresh.sum()
    over = (last - torch.clamp(first, min=width)).clamp(min=0).sum()
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    at = torch.arange(case["tokens"], device=table.device)
    b = torch.searchsorted(cu, at, right=True) - 1
    real, b = b < n, b.clamp(max=n - 1)
    pos = torch.where(real, held[b] + at - cu[b], 0)
    page = table[b, (pos // ps).clamp(max=width - 1)].long()
    slots = torch.where(real & (pos < width * ps) & (page >= 0), page * ps + pos % ps, -1)
    return {"kv_len": total.int(), "cu_new": cu.int(), "free_left": (top - wanted).clamp(min=0).int().view(1),
            "pages_short": ((wanted - top).clamp(min=0) + over).int().view(1), "positions": pos.int(), "slots": slots,
            "table": table, "free": free}


def _plain_rope(st, case):
    cos, sin = (st[k][st["positions"].long()][:, None] for k in ("cos", "sin"))
    half = case["rot"] // 2
    out = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
        if case["pairs"] == "halves":
            a, b, rest = y[..., :half], y[..., half:2 * half], y[..., 2 * half:]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
        else:
            a, b, rest = y[..., 0:2 * half:2], y[..., 1:2 * half:2], y[..., 2 * half:]
            y = torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)
        out.append(y.to(x.dtype))
    return {"q": out[0], "k": out[1]}


def _plain_store(st, case):
    d, ps, hk = case["d"], case["ps"], case["hk"]
    pages, lut = st["pages"].view(-1, hk, ps // 16, 18 * d), _pairs(st["pages"].device)
    page, row = st["slots"] // ps, st["slots"] % ps
    heads = torch.arange(hk, device=page.device)[None]
    at = (page[:, None], heads, (row // 16)[:, None])
    got = []
    for x, c, s in ((st["k"], 0, 16 * d), (st["v"], 8 * d, 17 * d)):
        codes, scales = _quantise(x)
        codes, raw = _pack(codes), scales.view(torch.uint8)
        for data, begin in ((codes, c), (raw, s)):
            byte = begin + (row % 16)[:, None, None] * data.shape[-1] + torch.arange(data.shape[-1], device=page.device)
            pages[tuple(a[..., None] for a in at) + (byte,)] = data
        got.append(_values(codes, scales, lut).to(x.dtype))
    return {"k": got[0], "v": got[1]}


def _plain_attend(st, case):
    d, ps, hk, hq = case["d"], case["ps"], case["hk"], case["hq"]
    q, table, kv = st["q"].float(), st["table"], st["kv_len"].long()
    n, group, most, dev = table.shape[0], hq // hk, case["queries"], q.device
    blocks = st["pages"].view(-1, hk, ps // 16, 18 * d)[table.clamp(min=0).long()]  # [n, pages, hk, blocks, bytes]
    lut = _pairs(dev)
    kc, vc, ks, vs = _parts(blocks, d)
    dense = lambda c, s: _values(c, s, lut).permute(0, 2, 1, 3, 4, 5).flatten(2, 4)  # noqa: E731  [n, hk, keys, d]
    cu = st["cu_q"].long()
    i = torch.arange(most, device=dev)[None]
    new = (cu[1:] - cu[:-1])[:, None]
    token = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)  # [n, most]
    rows = q[token].view(n, most, hk, group, d).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = rows @ dense(kc, ks).transpose(-1, -2) / math.sqrt(d)
    key = torch.arange(s.shape[-1], device=dev)
    pos = kv[:, None] - new + i  # of each query
    seen = (key < kv[:, None, None]).expand(n, most, -1)
    if case["causal"]:
        seen = seen & (key <= pos[..., None])
    if case["window"]:
        seen = seen & (key > pos[..., None] - case["window"])
    seen = seen[:, None].repeat_interleave(group, 2)
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    base = m.masked_fill(m == -math.inf, 0.0)
    p = torch.exp(s - base)
    total = p.sum(-1, keepdim=True)
    o = p @ dense(vc, vs) / total.masked_fill(total == 0, 1.0)
    lse = base + torch.log(total)
    pick = (i < new).nonzero(as_tuple=True)  # in the order of the tokens
    back = lambda x: x.unflatten(2, (most, group)).permute(0, 2, 1, 3, 4)[pick].flatten(1, 2)  # noqa: E731
    return {"out": back(o).to(st["q"].dtype), "lse": back(lse)[..., 0]}


_PLAIN = {"slots": _plain_slots, "rope": _plain_rope, "store": _plain_store, "attend": _plain_attend}


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    if case["op"] == "slots":
        return None  # whole numbers only
    st = {"case": case, "op": case["op"]}
    _PREPARE[case["op"]](st, case, torch.Generator(device="cuda").manual_seed(seed))
    return _EXACT[case["op"]](st, case)


def _exact_rope(st, case):
    rot = case["rot"]
    position = st["positions"].long()
    turn = torch.complex(st["cos"].double(), st["sin"].double())[position][:, None]
    got = {}
    for name, x, w in (("q", st["q"], st["wq"]), ("k", st["k"], st["wk"])):
        x = x.double()
        x = w.double() * x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6)
        z = x[..., :rot]
        z = z.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["pairs"] == "halves" else z.unflatten(-1, (rot // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
        z = z.transpose(-1, -2) if case["pairs"] == "halves" else z
        got[name] = torch.cat([z.flatten(-2), x[..., rot:]], -1)
    return got


def _exact_store(st, case):
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    got = {}
    for name in ("k", "v"):
        x = st[name].double().unflatten(-1, (case["d"] // GROUP, GROUP))
        s = (x.abs().amax(-1, keepdim=True) / 6).clamp(SCALE_MIN, SCALE_MAX).half().double()
        y = x.abs() / s
        high = torch.searchsorted(grid, y.contiguous()).clamp(1, 7)  # grid[high - 1] < y <= grid[high]
        low = high - 1
        down, up = y - grid[low], grid[high] - y
        pick = torch.where((down < up) | ((down == up) & (low % 2 == 0)), low, high)
        got[name] = (torch.copysign(grid[pick], x) * s).flatten(-2)
    return got


def _decode(raw, d):
    """bytes [..., d/2] -> values in 64 bits, from the layout's definition."""
    ch = torch.arange(d, device=raw.device)
    j, c, e = ch // 32, ch % 32 // 4, ch % 4
    nib = raw[..., (c * (d // 32) + j) * 2 + e // 2].long() >> (4 * (e % 2)) & 15
    mag, expo = nib & 1, nib >> 1 & 3
    value = torch.where(expo == 0, 0.5 * mag, (1 + 0.5 * mag) * 2.0 ** (expo.double() - 1))
    return torch.where(nib >= 8, -value, value.double())


def _exact_attend(st, case):
    d, ps, hk, group = case["d"], case["ps"], case["hk"], case["hq"] // case["hk"]
    new, kv = _lengths(case)
    outs, lses = [], []
    at = 0
    for b, (n, length) in enumerate(zip(new, kv)):
        pages = st["pages"][st["table"][b, :-(-length // ps)].long()].view(-1, hk, ps // 16, 18 * d)
        blocks = pages.transpose(0, 1).flatten(1, 2)  # [hk, blocks, bytes]
        full = []
        for c, s in ((0, 16 * d), (8 * d, 17 * d)):
            x = _decode(blocks[..., c:c + 8 * d].unflatten(-1, (16, d // 2)), d)
            scale = blocks[..., s:s + d].contiguous().view(torch.float16).double().unflatten(-1, (16, d // 32))
            full.append((x * scale.repeat_interleave(32, -1)).flatten(1, 2)[:, :length])
        q = st["q"][at:at + n].double().unflatten(1, (hk, group))
        pos = torch.arange(length - n, length, device="cuda")[:, None]
        key = torch.arange(length, device="cuda")[None]
        hide = torch.zeros(n, length, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hide |= key > pos
        if case["window"]:
            hide |= key <= pos - case["window"]
        for h in range(hk):
            s = torch.einsum("ngd,kd->ngk", q[:, h], full[0][h]) / math.sqrt(d)
            s = s.masked_fill(hide[:, None], -math.inf)
            lse = torch.logsumexp(s, -1) if length else torch.full((n, group), -math.inf, dtype=torch.float64, device="cuda")
            p = torch.exp(s - lse.masked_fill(lse == -math.inf, 0.0)[..., None])
            outs.append(torch.einsum("ngk,kd->ngd", p, full[1][h]))
            lses.append(lse)
        outs[-hk:] = [torch.cat(outs[-hk:], 1)]
        lses[-hk:] = [torch.cat(lses[-hk:], 1)]
        at += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


_EXACT = {"rope": _exact_rope, "store": _exact_store, "attend": _exact_attend}
