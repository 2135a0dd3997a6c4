"""Rows of a tile of prompts that are no rows (a group that does not divide 128, tokens behind a prompt's end) have no say in
those that are."""
import pytest

import serve_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def serve():
    from latency_barrier_free_gb300 import serve

    yield serve
    ref.leave_zeros()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def qkv(tokens, hq, hk, d, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [x.contiguous() for x in torch.randn(tokens, hq + 2 * hk, d, generator=gen, device="cuda").to(dtype).split([hq, hk, hk], 1)]


def leave_queries(prompts, by, d, max_len):
    """A call after which every row of the queries' shared memory holds `by` times normal values."""
    q, k, v = qkv(6000, 32, 4, d, torch.bfloat16, 1)
    prompts.attention(q * by, k, v, torch.empty_like(q), i32([0, 3000, 6000]), max_len=max_len)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("max_len", [1, 10 ** 6])  # either kernel
@pytest.mark.parametrize("group,d", [(3, 64), (5, 128), (7, 128), (12, 64)])
def test_what_another_call_left_changes_no_bit(serve, group, d, max_len, dtype):
    prompts, lengths = serve.PromptAttention(), [700, 390, 1]
    q, k, v = qkv(sum(lengths), 4 * group, 4, d, dtype)
    got = []
    for by in (0.0, 1000.0, float("nan"), float("inf")):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        leave_queries(prompts, by, d, max_len)
        prompts.attention(q, k, v, out, i32([0, 700, 1090, 1091]), max_len=max_len, lse=lse)
        got.append((out, lse))
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    assert prompts.status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("max_len", [1, 10 ** 6])
@pytest.mark.parametrize("hq,hk,d,window", [(8, 1, 128, 0), (14, 2, 64, 0), (4, 4, 64, 200)])
def test_a_neighbours_queries_change_no_bit(serve, hq, hk, d, window, max_len, dtype):
    prompts, (n, m) = serve.PromptAttention(), (471, 530)
    q, k, v = qkv(n + m, hq, hk, d, dtype)
    got = []
    for by in (1.0, 0.0, 1000.0, float("nan")):
        q2 = q.clone()
        q2[n:] *= by
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        prompts.attention(q2, k, v, out, i32([0, n, n + m]), max_len=max_len, window=window, lse=lse)
        got.append((out[:n], lse[:n]))
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    assert prompts.status() == 0


@pytest.mark.parametrize("max_len", [1, 10 ** 6])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("token", [0, 150, 333])
@pytest.mark.parametrize("what", ["key", "query"])
def test_keys_and_queries_that_are_infinite(serve, what, token, sign, max_len):
    """A score of +inf makes its row NaN or infinite; one of -inf has weight 0; a row with no other scores is one that sees no key."""
    n, d = 400, 64
    q, k, v = qkv(n, 2, 1, d, torch.bfloat16, 3)
    prompts, cu = serve.PromptAttention(), i32([0, n])
    (q if what == "query" else k)[token, :, 5] = sign * float("inf")
    out, lse = torch.empty_like(q), torch.empty(n, 2, device="cuda")
    prompts.attention(q, k, v, out, cu, max_len=max_len, lse=lse)
    assert prompts.status() == 0
    s = (q[:, :, None].double() * k[:, 0].double()).sum(-1).transpose(0, 1) / d ** 0.5  # [heads, queries, keys]
    s = s.masked_fill(torch.ones(n, n, device="cuda", dtype=torch.bool).triu(1), float("-inf"))
    high, none = (s == float("inf")).any(-1).T, (s == float("-inf")).all(-1).T
    assert (high | none).any()
    assert not torch.isfinite(out[high]).any() and not torch.isfinite(lse[high]).any()
    assert (out[none] == 0).all() and (lse[none] == float("-inf")).all()
    fine = ~(high | none)
    want = torch.einsum("hij,jd->ihd", s.softmax(-1), v[:, 0].double())[fine]
    mean = torch.einsum("hij,jd->ihd", s.softmax(-1), v[:, 0].double().abs())[fine]
    # a weight, and the result, to bfloat16; a score is a sum of 64 products below 20 in binary32, times 1/8: off by
    # 64 * 2 * 2^-24 * 64 * 20 / 8 = 1.2e-3 if all of them were, and were rounded the same way
    assert ((out[fine].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1.01 * (2.0 ** -8 + 2.4e-3) * mean).all()
    assert ((lse.double() - s.logsumexp(-1).T)[fine].abs() <= 1.3e-3).all()
