"""Cases of the serving operators around a prompt, an 8-bit cache and shared pages (latency_barrier_free_gb300/serve.py).

Next to the decode step's own work a serving program has: the attention of whole
prompts over their own keys and values (`prompt`); a key/value cache held in 8
bits, its write and what it stands for (`store8`), and the attention over it
(`attend8`); samples that share the pages of their prompt (`fork`); and what
follows when requests end, their pages given back and the rest moved to the
pool's low end (`tidy`).  A case names one of these and its sizes.  `run`
computes it in plain torch operations in 32 bits, or, with `own` set, by the
package's operators; `exact` computes it in 64 bits.

The 8-bit cache.  A page holds `ps` tokens (a multiple of 16) of every KV head:
bytes [head][block of 16 tokens][32 * d + 16].  A block of 16 tokens is K codes
(16 x d bytes), V codes (16 x d), the exponents of K and of V (a signed byte
each), 14 bytes that nothing uses.  A value is code * 2^exponent, a code is
e4m3.  The 16-byte piece p of a row r's codes lies in the 128-byte line that row
order gives, at p ^ (r & 7) within it for d = 128, at p ^ (r & 6) for d = 64
(two rows a line).  The exponent is the smallest that makes the block's largest
magnitude at most 448 units, within [-32, 32]; writing a block's first token
starts it anew, other tokens can only raise it, and then the codes that are
there are rounded to the new unit.
"""
import math
import random

import torch

own = False

LOW, HIGH, LARGEST = -32, 32, 448.0  # exponents, and the largest code


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # a few short chat turns at once, odd groups of 7 heads, small heads: latency
        {"name": "prompt 5 short", "op": "prompt", "requests": 5, "longest": 96, "hq": 14, "hk": 2, "d": 64,
         "dtype": "bf16", "causal": True, "window": 0},
        # ragged prompts on one of eight tensor-parallel ranks, sliding window, binary16
        {"name": "prompt 12 ragged fp16", "op": "prompt", "requests": 12, "longest": 2048, "hq": 8, "hk": 1, "d": 128,
         "dtype": "fp16", "causal": True, "window": 1000},
        # two long documents, all heads of the [B, 8192] model
        {"name": "prompt 2 long", "op": "prompt", "requests": 2, "longest": 8192, "hq": 64, "hk": 8, "d": 128,
         "dtype": "bf16", "causal": True, "window": 0},
        # the cache write of a decode step, and what the touched blocks stand for
        {"name": "store8 16 tokens", "op": "store8", "requests": 16, "queries": 1, "longest": 4096, "hk": 8, "d": 128,
         "ps": 64, "dtype": "bf16"},
        # the cache write of prompts that continue what is there
        {"name": "store8 4 prompts", "op": "store8", "requests": 4, "queries": 8192, "longest": 16384, "hk": 8, "d": 128,
         "ps": 64, "dtype": "bf16"},
        # one request on one tensor-parallel rank: latency
        {"name": "attend8 1 x 2000", "op": "attend8", "requests": 1, "queries": 1, "longest": 2000, "hq": 8, "hk": 1,
         "d": 128, "ps": 64, "causal": True, "window": 0},
        # a decode batch of 64 ragged requests, all heads, some padding
        {"name": "attend8 64 ragged", "op": "attend8", "requests": 64, "queries": 1, "longest": 16384, "hq": 64, "hk": 8,
         "d": 128, "ps": 64, "causal": True, "window": 0},
        # prompts in chunks on top of what the cache already holds
        {"name": "attend8 prompt chunks", "op": "attend8", "requests": 3, "queries": 1024, "longest": 8192, "hq": 64,
         "hk": 8, "d": 128, "ps": 64, "causal": True, "window": 0},
        # one prompt sampled eight times: latency
        {"name": "fork 1 into 8", "op": "fork", "requests": 1, "samples": 8, "longest": 1000, "hk": 1, "d": 128, "ps": 64},
        # a batch of prompts, each sampled eight times, whole pages of all heads
        {"name": "fork 32 into 8", "op": "fork", "requests": 32, "samples": 8, "longest": 4096, "hk": 8, "d": 128, "ps": 64},
        # a few requests end, odd sizes
        {"name": "tidy 9 requests", "op": "tidy", "requests": 9, "longest": 700, "hk": 1, "d": 64, "ps": 16, "moves": 64},
        # a large pool after much traffic, every fourth request ends
        {"name": "tidy 500 requests", "op": "tidy", "requests": 500, "longest": 16384, "hk": 2, "d": 128, "ps": 64,
         "moves": 8192},
    ]


def _log(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "store8", "attend8", "attend8", "attend8", "fork", "tidy"])
    d, ps = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    hk, group = _log(rng, 1, 8), rng.choice([1, 2, 4, 5, 7, 8, 8, 16])
    hq = hk * min(group, 64 // hk)
    if op == "prompt":
        causal = rng.random() < 0.8
        longest = _log(rng, 1, 8192 if causal else 4096)
        return {"op": op, "requests": _log(rng, 1, max(1, min(64, (16384 if causal else 8192) // longest))), "longest": longest,
                "hq": hq, "hk": hk, "d": rng.choice([d, d, d, 80, 96]), "dtype": rng.choice(["bf16", "fp16"]),
                "causal": causal, "window": rng.choice([0, 0, 0, _log(rng, 16, 4096)])}
    if op == "store8":
        queries = rng.choice([1, 1, _log(rng, 2, 8192)])
        return {"op": op, "requests": _log(rng, 1, max(1, min(256, 32768 // queries))), "queries": queries,
                "longest": queries + _log(rng, 1, 8192), "hk": hk, "d": d, "ps": ps,
                "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "attend8":
        queries = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 1024)])
        most = 2 ** 20 if queries == 1 else 2 ** 18 if queries <= 8 else 24576  # keys of all requests together
        longest = _log(rng, max(queries, 16), 131071 if queries <= 8 else 8192)
        return {"op": op, "requests": _log(rng, 1, max(1, min(64, most // longest))), "queries": queries,
                "longest": longest, "hq": hq, "hk": hk, "d": d, "ps": ps,
                "causal": rng.random() < 0.9, "window": rng.choice([0, 0, 0, _log(rng, 16, 4096)])}
    if op == "fork":
        return {"op": op, "requests": _log(rng, 1, 32), "samples": rng.randint(1, 8), "longest": _log(rng, 1, 4096), "hk": hk,
                "d": d, "ps": ps}
    return {"op": op, "requests": _log(rng, 1, 500), "longest": _log(rng, ps, 16384), "hk": min(hk, 2), "d": d,
            "ps": max(ps, 32), "moves": _log(rng, 16, 8192)}


def _lengths(case):
    """Tokens of each request that are new, and all of its tokens; they go by the case alone, so that work() knows them."""
    rng = random.Random("%s %d %d" % (case["op"], case["requests"], case["longest"]))
    n, most = case["requests"], case.get("queries", case["longest"])
    new = [most] + [_log(rng, 1, most) for _ in range(n - 1)]
    if case["op"] in ("prompt", "fork", "tidy"):
        if n >= 4:
            new[-1], new[-2] = 0, 1  # padding of a batch, and the shortest prompt there is
        return new, new
    kv = [case["longest"]] + [max(q, _log(rng, min(16, case["longest"]), case["longest"])) for q in new[1:]]
    if n >= 16:
        kv[-1], kv[-2] = 0, 1  # a request whose rows see no key, and one whose first token this is
        new[-2] = 1
        if case["op"] == "store8":
            new[-1] = 0
    return new, kv


def _ends(b):
    """Whether request b of a `tidy` case ends."""
    return b % 4 == 1 or b % 16 == 4


def _page_bytes(case):
    return case["hk"] * (case["ps"] // 16) * (32 * case["d"] + 16)


def work(case):
    new, kv = _lengths(case)
    d, hk = case["d"], case["hk"]
    if case["op"] == "store8":  # values in, codes out and in, values out
        size, t = {"bf16": 2, "fp32": 4}[case["dtype"]], sum(new)
        return {"bytes": 2 * t * hk * d * (2 * size + 2) + 8 * t, "flops": 4 * t * hk * d}
    ps = case.get("ps", 16)
    if case["op"] == "fork":
        entries = sum(-(-x // ps) for x in kv) * case["samples"]
        tails = sum(x % ps != 0 for x in kv) * case["samples"]
        return {"bytes": 12 * entries + 2 * tails * _page_bytes(case), "flops": 0}
    if case["op"] == "tidy":
        held, pool = [-(-x // ps) for x in kv], _pool(case)
        used = sum(h for b, h in enumerate(held) if not _ends(b))
        moves = min(case["moves"], used * (pool - used) // pool)  # as many as a random order is expected to need
        return {"bytes": 16 * pool + 8 * sum(held) + 2 * moves * _page_bytes(case), "flops": 0}
    pairs = keys = 0
    for n, length in zip(new, kv):
        first = length
        for i in range(n):
            end = min(length, max(0, length - n + i + 1)) if case["causal"] else length
            begin = max(0, length - n + i + 1 - case["window"]) if case["window"] else 0
            pairs += max(0, end - begin)
            first = min(first, begin)
        keys += length - first
    rows = sum(new) * case["hq"]
    if case["op"] == "prompt":
        return {"bytes": 4 * d * (keys * hk + rows) + 4 * rows, "flops": 4 * pairs * case["hq"] * d}
    return {"bytes": 2 * keys * hk * d + 4 * rows * (d + 1), "flops": 4 * pairs * case["hq"] * d}


def _pool(case):
    """Pages of a `tidy` case: half again what its requests hold."""
    return sum(-(-x // case["ps"]) for x in _lengths(case)[1]) * 3 // 2 + 8


# ----------------------------------------------------- the 8-bit cache, plain --
def _at(d, device):
    """[16, d]: the byte of each row and channel in a block's codes."""
    row, ch = torch.arange(16, device=device)[:, None], torch.arange(d, device=device)[None]
    byte = row * d + ch
    turn = row & 7 if d == 128 else row & 6
    return byte // 128 * 128 + ((byte // 16 % 8) ^ turn) * 16 + byte % 16


def _exponent(most):
    """The smallest e with most <= 448 * 2^e, within the limits."""
    m, e = torch.frexp(most)  # most = m * 2^e, m in [.5, 1); 448 = .875 * 2^9
    return torch.where(most > 0, e - 9 + (m > 0.875), LOW).clamp(LOW, HIGH)


def _two(e):
    """2^e, exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _codes(x, e):
    """x over 2^e as e4m3 bytes, saturating."""
    y = (torch.nan_to_num(x.float(), nan=0.0) * _two(-e)).clamp(-LARGEST, LARGEST)
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _blocks(pages, case):
    return pages.view(-1, case["hk"], case["ps"] // 16, 32 * case["d"] + 16)


def _fill(pages, case, gen):
    """Keys and values of normal size in every block; every head has a size of its own, as real ones do."""
    d, hk, ps = case["d"], case["hk"], case["ps"]
    blocks, at = _blocks(pages, case), _at(d, pages.device).flatten()
    step = max(1, (1 << 26) // (hk * ps * d))
    for begin in range(0, blocks.shape[0], step):
        part = blocks[begin:begin + step]
        for n in range(2):
            x = torch.randn(part.shape[:3] + (16 * d,), generator=gen, device=pages.device)
            x *= torch.linspace(0.5, 2.0, hk, device=pages.device)[:, None, None] * (1.0 if n == 0 else 0.3)
            e = _exponent(x.abs().amax(-1))
            part[..., n * 16 * d + at] = _codes(x, e[..., None])
            part[..., 32 * d + n] = e.to(torch.int8).view(torch.uint8)


# ---------------------------------------------------------------- prepare --
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case, "op": case["op"]}
    _PREPARE[case["op"]](st, case, gen)
    if own:  # the handles that a serving program keeps
        from latency_barrier_free_gb300 import serve

        if case["op"] == "prompt":
            st["prompts"] = serve.PromptAttention()
        else:
            st["cache"] = serve.KvCache8(st["pages"], case["ps"], case["hk"], case["d"])
    return st


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _zeros(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


def _running(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _prepare_prompt(st, case, gen):
    new, _ = _lengths(case)
    t, hq, hk, d = sum(new), case["hq"], case["hk"], case["d"]
    qkv = torch.randn(t, hq + 2 * hk, d, generator=gen, device="cuda").to(_TYPES[case["dtype"]])  # the packed projection
    q, k, v = qkv.split([hq, hk, hk], 1)
    st.update(q=q, k=k, v=v, cu=_ints(_running(new)), out=torch.empty(t, hq, d, dtype=q.dtype, device="cuda"),
              lse=torch.empty(t, hq, device="cuda"))


def _tables(counts, pool, gen, spare=0):
    """Pages in the order of past traffic: the requests' tables (and `spare` empty rows), and the stack of free pages."""
    width = max(max(counts), 1)
    order = torch.randperm(pool, generator=gen, device="cuda").int()
    table = torch.full((len(counts) + spare, width), -1, dtype=torch.int32, device="cuda")
    inside = torch.arange(width, device="cuda")[None] < torch.tensor(counts, device="cuda")[:, None]
    table[:len(counts)][inside] = order[:sum(counts)]
    free = _zeros(pool)
    free[:pool - sum(counts)] = order[sum(counts):]
    return table, free, _ints([pool - sum(counts)])


def _prepare_store8(st, case, gen):
    new, kv = _lengths(case)
    ps, hk, d, t = case["ps"], case["hk"], case["d"], sum(new)
    dt = _TYPES[case["dtype"]]
    held = [-(-n // ps) for n in kv]
    pool = sum(held) + 4
    table, _, _ = _tables(held, pool, gen)
    b = torch.repeat_interleave(torch.arange(len(new), device="cuda"), torch.tensor(new, device="cuda"))
    first = torch.tensor([k - n for k, n in zip(kv, new)], device="cuda")
    pos = first[b] + torch.arange(t, device="cuda") - torch.tensor(_running(new)[:-1], device="cuda")[b]
    slots = table[b, pos // ps].long() * ps + pos % ps
    # what the touched blocks hold before the first new token, too
    before = [(f % 16 if n else 0) for f, n in zip(first.tolist(), new)]
    ob = torch.repeat_interleave(torch.arange(len(new), device="cuda"), torch.tensor(before, device="cuda"))
    opos = first[ob] // 16 * 16 + torch.arange(sum(before), device="cuda") - torch.tensor(_running(before)[:-1], device="cuda")[ob]
    old = table[ob, opos // ps].long() * ps + opos % ps
    size = torch.linspace(0.5, 2.0, hk, device="cuda")[:, None]
    pages = torch.zeros(pool, _page_bytes(case), dtype=torch.uint8, device="cuda")
    _fill(pages, case, gen)
    read = torch.cat([slots, old])
    st.update(k=(1.5 * torch.randn(t, hk, d, generator=gen, device="cuda") * size).to(dt),
              v=(0.3 * torch.randn(t, hk, d, generator=gen, device="cuda") * size).to(dt), slots=slots, read=read, pages=pages,
              k_out=torch.empty(read.numel(), hk, d, dtype=dt, device="cuda"),
              v_out=torch.empty(read.numel(), hk, d, dtype=dt, device="cuda"))


def _prepare_attend8(st, case, gen):
    new, kv = _lengths(case)
    ps, t = case["ps"], sum(new)
    held = [-(-n // ps) for n in kv]
    pool = sum(held) + 4
    table, _, _ = _tables(held, pool, gen)
    pages = torch.zeros(pool, _page_bytes(case), dtype=torch.uint8, device="cuda")
    _fill(pages, case, gen)
    q = torch.randn(t, case["hq"], case["d"], generator=gen, device="cuda").bfloat16()
    st.update(q=q, cu_q=_ints(_running(new)), kv_len=_ints(kv), table=table, pages=pages, out=torch.empty_like(q),
              lse=torch.empty(t, case["hq"], device="cuda"))


def _contents(pool, case, gen):
    return torch.randint(0, 256, (pool, _page_bytes(case)), dtype=torch.uint8, generator=gen, device="cuda")


def _prepare_fork(st, case, gen):
    _, kv = _lengths(case)
    ps, n, forks = case["ps"], case["requests"], case["requests"] * case["samples"]
    held = [-(-x // ps) for x in kv]
    pool = sum(held) + forks + 8
    table, free, count = _tables(held, pool, gen, forks)
    out = {"kv_len": _zeros(n + forks), "shared": _zeros(pool), "copy_from": _zeros(forks), "copy_to": _zeros(forks),
           "free_left": _zeros(1), "pages_short": _zeros(1)}
    st.update(seq_len=_ints(kv + [0] * forks), table=table, free=free, free_count=count, shared=_zeros(pool),
              source=_ints([i // case["samples"] for i in range(forks)]), target=_ints(list(range(n, n + forks))),
              pages=_contents(pool, case, gen), out=out)


def _prepare_tidy(st, case, gen):
    _, kv = _lengths(case)
    ps, n, pool = case["ps"], case["requests"], _pool(case)
    held = [-(-x // ps) for x in kv]
    table, free, count = _tables(held, pool, gen)
    shared = _zeros(pool)
    for b in range(5, n, 8):  # samples of one prompt: this request begins with the whole pages of the one before
        common = min(kv[b], kv[b - 1]) // ps
        if common:
            pages = table[b, :common].clone()
            table[b, :common] = table[b - 1, :common]
            shared[table[b - 1, :common].long()] += 1
            free[count.long() + torch.arange(common, device="cuda")] = pages
            count += common
    new = [-1 if _ends(b) else 1 for b in range(n)]
    out = {"kv_len": _zeros(n), "left": _zeros(pool), "mid": _zeros(1), "table": torch.empty_like(table), "free": _zeros(pool),
           "shared": _zeros(pool), "free_left": _zeros(1), "moved": _zeros(pool), "move_from": _zeros(case["moves"]),
           "move_to": _zeros(case["moves"]), "move_count": _zeros(1)}
    st.update(seq_len=_ints(kv), new_len=_ints(new), table=table, free=free, free_count=count, shared=shared,
              pages=_contents(pool, case, gen), out=out)


_PREPARE = {"prompt": _prepare_prompt, "store8": _prepare_store8, "attend8": _prepare_attend8, "fork": _prepare_fork,
            "tidy": _prepare_tidy}


# -------------------------------------------------------------------- run --
def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state, state["case"])


def _own_prompt(st, case):
    st["prompts"].attention(st["q"], st["k"], st["v"], st["out"], st["cu"], max_len=case["longest"], causal=case["causal"],
                            window=case["window"], lse=st["lse"])
    return {"out": st["out"], "lse": st["lse"]}


def _own_store8(st, case):
    st["cache"].append(st["k"], st["v"], st["slots"])
    st["cache"].read(st["read"], st["k_out"], st["v_out"])
    return {"k": st["k_out"], "v": st["v_out"]}


def _own_attend8(st, case):
    st["cache"].attention(st["q"], st["out"], st["cu_q"], st["kv_len"], st["table"], max_q=case["queries"],
                          max_kv=case["longest"], causal=case["causal"], window=case["window"], lse=st["lse"])
    return {"out": st["out"], "lse": st["lse"]}


def _own_fork(st, case):
    from latency_barrier_free_gb300 import serve

    o = st["out"]
    serve.pages_fork(st["seq_len"], st["source"], st["target"], st["table"], st["free"], st["free_count"], st["shared"],
                     case["ps"], kv_len=o["kv_len"], shared_out=o["shared"], copy_from=o["copy_from"],
                     copy_to=o["copy_to"], free_left=o["free_left"], pages_short=o["pages_short"])
    st["cache"].copy(o["copy_from"], o["copy_to"])
    return dict(o, table=st["table"], pages=st["pages"])


def _own_tidy(st, case):
    from latency_barrier_free_gb300 import serve

    o = st["out"]
    serve.pages_release(st["seq_len"], st["new_len"], st["table"], st["free"], st["free_count"], st["shared"], case["ps"],
                        kv_len=o["kv_len"], shared_out=o["left"], free_left=o["mid"])
    serve.pages_compact(o["kv_len"], st["table"], st["free"], o["mid"], o["left"], case["ps"], table_out=o["table"],
                        free_out=o["free"], shared_out=o["shared"], free_left=o["free_left"], moved=o["moved"],
                        move_from=o["move_from"], move_to=o["move_to"], move_count=o["move_count"])
    st["cache"].copy(o["move_from"], o["move_to"])
    return dict(o, pages=st["pages"])


_OWN = {"prompt": _own_prompt, "store8": _own_store8, "attend8": _own_attend8, "fork": _own_fork, "tidy": _own_tidy}


def _softmax(s, seen, values):
    """Weighted sums of values, and the log-sum-exp, over the keys that are seen."""
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    base = m.masked_fill(m == -math.inf, 0.0)
    p = torch.exp(s - base)
    total = p.sum(-1, keepdim=True)
    o = p @ values / total.masked_fill(total == 0, 1.0)
    return o, (base + torch.log(total))[..., 0]


def _plain_prompt(st, case):
    hk, group, n = case["hk"], case["hq"] // case["hk"], case["longest"]
    q, k, v = (st[x].float() for x in "qkv")
    cu = st["cu"].long()
    at = torch.arange(n, device=q.device)
    token = (cu[:-1, None] + at).clamp(max=q.shape[0] - 1)  # [requests, n]
    length = cu[1:] - cu[:-1]
    seen = (at < length[:, None, None]).expand(-1, n, -1)
    if case["causal"]:
        seen = seen & (at[:, None] >= at)
    if case["window"]:
        seen = seen & (at[:, None] - at < case["window"])
    outs, lses = [], []
    for h in range(hk):  # a KV head's scores at a time: those of all would not fit
        rows = q[token][:, :, h * group:(h + 1) * group].transpose(1, 2)  # [requests, group, n, d]
        s = rows @ k[token][:, None, :, h].transpose(-1, -2) / math.sqrt(case["d"])
        o, lse = _softmax(s, seen[:, None], v[token][:, None, :, h])
        outs.append(o)
        lses.append(lse)
    pick = (at < length[:, None]).nonzero(as_tuple=True)  # in the order of the tokens
    o = torch.cat(outs, 1).transpose(1, 2)[pick]
    return {"out": o.to(st["q"].dtype), "lse": torch.cat(lses, 1).transpose(1, 2)[pick]}


def _plain_store8(st, case):
    d, hk, ps = case["d"], case["hk"], case["ps"]
    blocks, at = _blocks(st["pages"], case), _at(case["d"], st["pages"].device)
    flat = blocks.transpose(1, 2).reshape(-1, hk, 32 * d + 16)  # [pages * blocks, heads, bytes], a copy
    b, row = st["slots"] // 16, st["slots"] % 16
    fresh = torch.zeros(flat.shape[0], dtype=torch.bool, device=b.device)
    fresh[b[row == 0]] = True
    touched = torch.zeros_like(fresh)
    touched[b] = True
    for n, x in enumerate((st["k"].float(), st["v"].float())):
        e = _exponent(x.abs().amax(-1)).to(torch.int32)  # [tokens, heads]
        old = flat[..., 32 * d + n].view(torch.int8).int()
        most = torch.where(fresh[:, None], torch.full_like(old, LOW), old)
        most = torch.where(touched[:, None], most.scatter_reduce(0, b[:, None].expand_as(e), e, "amax"), old)
        codes = flat[..., n * 16 * d:(n + 1) * 16 * d]
        # what is there, in the new unit
        again = _codes(_values(codes), (most - old).clamp(min=0)[..., None])
        codes = torch.where((most > old)[..., None], again, codes)
        heads = torch.arange(hk, device=b.device)
        codes[b[:, None, None], heads[:, None], at[row][:, None]] = _codes(x, most[b][..., None])
        flat[..., n * 16 * d:(n + 1) * 16 * d] = codes
        flat[..., 32 * d + n] = most.to(torch.int8).view(torch.uint8)
    blocks.copy_(flat.view(-1, ps // 16, hk, 32 * d + 16).transpose(1, 2))
    got = []
    b, row = st["read"] // 16, st["read"] % 16
    for n in range(2):
        codes = flat[b[:, None, None], torch.arange(hk, device=b.device)[:, None], n * 16 * d + at[row][:, None]]
        e = flat[..., 32 * d + n].view(torch.int8).int()[b]
        got.append((_values(codes) * _two(e)[..., None]).to(st["k"].dtype))
    return {"k": got[0], "v": got[1]}


def _dense(pages, table, case):
    """Keys and values [requests, heads, tokens, d] of the tables' pages in 32 bits."""
    d = case["d"]
    blocks = _blocks(pages, case)[table.clamp(min=0).long()].transpose(1, 2).flatten(2, 3)  # [n, hk, blocks, bytes]
    at = _at(d, pages.device).flatten()
    got = []
    for n in range(2):
        e = blocks[..., 32 * d + n].contiguous().view(torch.int8).int()
        got.append((_values(blocks[..., n * 16 * d + at]) * _two(e)[..., None]).unflatten(-1, (16, d)).flatten(2, 3))
    return got


def _plain_attend8(st, case):
    hk, hq = case["hk"], case["hq"]
    q, table, kv = st["q"].float(), st["table"], st["kv_len"].long()
    n, group, most, dev = table.shape[0], hq // hk, case["queries"], q.device
    keys, values = _dense(st["pages"], table, case)
    cu = st["cu_q"].long()
    i = torch.arange(most, device=dev)[None]
    new = (cu[1:] - cu[:-1])[:, None]
    token = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)  # [n, most]
    rows = q[token].view(n, most, hk, group, case["d"]).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = rows @ keys.transpose(-1, -2) / math.sqrt(case["d"])
    key = torch.arange(s.shape[-1], device=dev)
    pos = kv[:, None] - new + i  # of each query
    seen = (key < kv[:, None, None]).expand(n, most, -1)
    if case["causal"]:
        seen = seen & (key <= pos[..., None])
    if case["window"]:
        seen = seen & (key > pos[..., None] - case["window"])
    o, lse = _softmax(s, seen[:, None].repeat_interleave(group, 2), values)
    pick = (i < new).nonzero(as_tuple=True)  # in the order of the tokens
    back = lambda x: x.unflatten(2, (most, group)).permute(0, 2, 1, 3, 4)[pick].flatten(1, 2)  # noqa: E731
    return {"out": back(o).to(st["q"].dtype), "lse": back(lse[..., None])[..., 0]}


def _plain_fork(st, case):
    ps, table, free, o = case["ps"], st["table"], st["free"], st["out"]
    source, target = st["source"].long(), st["target"].long()
    width, pool = table.shape[1], free.numel()
    length = st["seq_len"][source].long()
    full = (length // ps).clamp(max=width)[:, None]
    rows, col = table[source], torch.arange(width, device=table.device)
    valid = (rows >= 0) & (rows < pool)
    o["shared"].copy_(st["shared"])
    o["shared"].view(-1).scatter_add_(0, rows.clamp(0, pool - 1).flatten().long(), (valid & (col < full)).flatten().int())
    # the page that a request has not filled becomes a page of the sample's own
    last = (col == full) & (length % ps != 0)[:, None] & valid
    needs = last.any(1)
    page = torch.where(needs, rows.gather(1, full.clamp(max=width - 1))[:, 0], -1)
    rank, count = needs.cumsum(0) - 1, st["free_count"].long()
    given = torch.where(needs & (rank < count), free[(count - 1 - rank).clamp(0, pool - 1)], -1)
    held = ((length + ps - 1) // ps)[:, None]
    table[target] = torch.where(last, given[:, None], torch.where(col < held, rows, table[target]))
    o["kv_len"].copy_(st["seq_len"])
    o["kv_len"][target] = length.int()
    o["copy_from"].copy_(torch.where(given >= 0, page, -1))
    o["copy_to"].copy_(given)
    o["free_left"].copy_((count - needs.sum()).clamp(min=0))
    o["pages_short"].copy_((needs.sum() - count).clamp(min=0))
    some = (given >= 0).nonzero()[:, 0]
    st["pages"][given[some].long()] = st["pages"][page[some].long()]
    return dict(o, table=table, pages=st["pages"])


def _plain_tidy(st, case):
    ps, table, free, o = case["ps"], st["table"], st["free"], st["out"]
    width, pool = table.shape[1], free.numel()
    col, page = torch.arange(width, device=table.device), torch.arange(pool, device=table.device)
    length, ends = st["seq_len"].long(), st["new_len"] < 0
    # release: holders that end; a page without any goes back, in the order of the pages
    drop = ends[:, None] & (col < ((length + ps - 1) // ps)[:, None]) & (table >= 0) & (table < pool)
    drops = torch.zeros(pool, dtype=torch.int64, device=table.device)
    drops.scatter_add_(0, table.clamp(0, pool - 1).flatten().long(), drop.flatten().long())
    back = drops > st["shared"]
    o["left"].copy_(torch.where(back, 0, st["shared"] - drops))
    rank, count = back.cumsum(0) - 1, st["free_count"].long()
    spare = torch.cat([free, free.new_zeros(1)])
    spare.scatter_(0, torch.where(back & (count + rank < pool), count + rank, pool), page.int())
    free.copy_(spare[:pool])
    mid = (count + back.sum()).clamp(max=pool)
    o["mid"].copy_(mid)
    o["kv_len"].copy_(torch.where(ends, 0, st["seq_len"]))
    # compact: the highest used pages to the lowest free ones
    spare = torch.zeros(pool + 1, dtype=torch.bool, device=table.device)
    spare[torch.where(page < mid, free.long(), pool)] = True
    is_free = spare[:pool]
    hole = is_free.long().cumsum(0) - 1  # rank from below
    used = (~is_free).long().flip(0).cumsum(0).flip(0) - 1  # rank from above
    total = (~is_free).sum()
    moves = (is_free & (page < total)).sum().clamp(max=case["moves"])
    leaves, gets = ~is_free & (used < moves), is_free & (hole < moves)
    lists = []
    for sel, rank in ((leaves, used), (gets, hole)):
        x = torch.full((case["moves"] + 1,), -1, dtype=torch.int64, device=table.device)
        x.scatter_(0, torch.where(sel, rank, case["moves"]), page)
        lists.append(x[:case["moves"]])
    source, target = lists
    moved = torch.where(is_free, -1, page)
    some = (source >= 0).nonzero()[:, 0]
    source, target = source[some], target[some]
    moved[source] = target
    o["moved"].copy_(moved)
    o["move_from"].copy_(lists[0])
    o["move_to"].copy_(lists[1])
    o["move_count"].copy_(moves)
    o["shared"].copy_(o["left"])
    o["shared"][target] = o["left"][source]
    o["shared"][source] = 0
    live = (col < ((o["kv_len"].long() + ps - 1) // ps)[:, None]) & (table >= 0) & (table < pool)
    o["table"].copy_(torch.where(live, moved[table.clamp(0, pool - 1).long()].int(), table))
    # the next page from the stack is the lowest
    now_free = (is_free & ~gets) | leaves
    rank = now_free.long().cumsum(0) - 1
    x = torch.cat([o["free"], o["free"].new_zeros(1)])
    x.scatter_(0, torch.where(now_free, now_free.sum() - 1 - rank, pool), page.int())
    o["free"].copy_(x[:pool])
    o["free_left"].copy_(now_free.sum())
    st["pages"][target] = st["pages"][source]
    return dict(o, pages=st["pages"])


_PLAIN = {"prompt": _plain_prompt, "store8": _plain_store8, "attend8": _plain_attend8, "fork": _plain_fork,
          "tidy": _plain_tidy}


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    if case["op"] in ("fork", "tidy"):
        return None  # whole numbers only
    if work(case)["flops"] > 4e12:
        return None
    st = {"case": case, "op": case["op"]}
    _PREPARE[case["op"]](st, case, torch.Generator(device="cuda").manual_seed(seed))
    return _EXACT[case["op"]](st, case)


def _exact_rows(q, k, v, pos, case):
    """q [n, group, d] at positions pos [n, 1], keys and values [length, d], all in 64 bits."""
    length = k.shape[0]
    key = torch.arange(length, device=q.device)[None]
    hide = torch.zeros(q.shape[0], length, dtype=torch.bool, device=q.device)
    if case["causal"]:
        hide |= key > pos
    if case["window"]:
        hide |= key <= pos - case["window"]
    if length == 0:
        return torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    s = torch.einsum("ngd,kd->ngk", q, k) / math.sqrt(case["d"])
    s = s.masked_fill(hide[:, None], -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse.masked_fill(lse == -math.inf, 0.0)[..., None])
    return torch.einsum("ngk,kd->ngd", p, v), lse


def _exact_prompt(st, case):
    new, _ = _lengths(case)
    hk = case["hk"]
    outs, lses, at = [], [], 0
    for n in new:
        q, k, v = (st[x][at:at + n].double() for x in "qkv")
        pos = torch.arange(n, device="cuda")[:, None]
        parts = []
        for rows in torch.arange(n, device="cuda").split(1024) if n else []:  # a stretch of queries and a head at a time
            got = [_exact_rows(q[rows].unflatten(1, (hk, -1))[:, h], k[:, h], v[:, h], pos[rows], case) for h in range(hk)]
            parts.append((torch.cat([o for o, _ in got], 1), torch.cat([x for _, x in got], 1)))
        outs += [o for o, _ in parts]
        lses += [x for _, x in parts]
        at += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _power(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_parts(blocks, d):
    """codes' values and exponents of blocks [..., bytes], from the layout's definition."""
    row, ch = torch.arange(16, device=blocks.device)[:, None], torch.arange(d, device=blocks.device)[None]
    line, piece = row * d // 128, row * d % 128 // 16 + ch // 16
    byte = 128 * line + 16 * (piece ^ (row % 8 if d == 128 else row % 8 - row % 2)) + ch % 16
    got = []
    for n in range(2):
        c = blocks[..., n * 16 * d:(n + 1) * 16 * d][..., byte].long()
        mag, ex = c % 8, c // 8 % 16
        value = torch.where(ex == 0, mag * 2.0 ** -9, (8 + mag) * _power(ex - 10))
        e = blocks[..., 32 * d + n].long()
        got.append((torch.where(c >= 128, -value, value), torch.where(e >= 128, e - 256, e)))
    return got


def _exact_round(y):
    """y in 64 bits to the nearest e4m3, ties to even, saturating."""
    m = y.abs().clamp(max=448.0)
    _, e = torch.frexp(m)
    step = _power(torch.clamp(e - 1, min=-6) - 3)
    return torch.copysign(torch.round(m / step) * step, y)


def _exact_store8(st, case):
    d, hk, ps = case["d"], case["hk"], case["ps"]
    parts = _exact_parts(_blocks(st["pages"], case).transpose(1, 2).reshape(-1, hk, 32 * d + 16), d)
    b, row = st["slots"] // 16, st["slots"] % 16
    anew = torch.zeros(parts[0][1].shape[0], dtype=torch.bool, device=b.device).index_fill(0, b[row == 0], True)
    got = {}
    for (value, e), name in zip(parts, "kv"):
        x = st[name].double()
        most = torch.zeros(e.shape, dtype=torch.float64, device=b.device)
        most = most.scatter_reduce(0, b[:, None].expand(-1, hk), x.abs().amax(-1), "amax")
        want = torch.ceil(torch.log2((most / 448.0).clamp(min=2.0 ** -40))).clamp(LOW, HIGH).long()
        want = torch.where((most > 448.0 * _power(want)) & (want < HIGH), want + 1, want)
        want = torch.where((most <= 448.0 * _power(want - 1)) & (want > LOW), want - 1, want)
        written = torch.zeros_like(anew).index_fill(0, b, True)[:, None]
        now = torch.where(written, torch.where(anew[:, None], want, torch.maximum(want, e)), e)
        value = _exact_round(value * _power((e - now).clamp(max=0))[..., None, None]) * _power(now)[..., None, None]
        unit = _power(now[b])[..., None]
        value[b, :, row] = _exact_round(x / unit) * unit
        got[name] = value[st["read"] // 16, :, st["read"] % 16]
    return got


def _exact_attend8(st, case):
    d, hk, ps = case["d"], case["hk"], case["ps"]
    new, kv = _lengths(case)
    outs, lses, at = [], [], 0
    for b, (n, length) in enumerate(zip(new, kv)):
        pages = _blocks(st["pages"][st["table"][b, :-(-length // ps)].long()], case)
        full = [(v * _power(e)[..., None, None]).transpose(0, 1).flatten(1, 3)[:, :length]
                for v, e in _exact_parts(pages, d)]
        q = st["q"][at:at + n].double().unflatten(1, (hk, -1))
        pos = torch.arange(length - n, length, device="cuda")[:, None]
        got = [_exact_rows(q[:, h], full[0][h], full[1][h], pos, case) for h in range(hk)]
        outs.append(torch.cat([o for o, _ in got], 1))
        lses.append(torch.cat([x for _, x in got], 1))
        at += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


_EXACT = {"prompt": _exact_prompt, "store8": _exact_store8, "attend8": _exact_attend8}
