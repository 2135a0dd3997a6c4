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
