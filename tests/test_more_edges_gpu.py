"""The prompts' attention and the 8-bit cache where waits run out, workspaces are shared and tensors are on other streams."""
import ctypes

import numpy as np
import pytest

import serve_ref as ref
from test_serve_edges_gpu import arguments, impatient  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def serve():
    from latency_barrier_free_gb300 import serve

    yield serve
    ref.leave_zeros()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# one prompt that is cut into runs (few segments, long), many that are dealt out, and short ones
@pytest.mark.parametrize("lengths,hq,hk,d", [([4000], 8, 1, 128), ([700, 30, 900, 0, 5] * 6, 16, 4, 64), ([20, 9], 4, 2, 128)])
@pytest.mark.parametrize("max_len", [1, 10 ** 6])  # either kernel
def test_after_a_wait_ran_out_the_next_prompt_is_right(serve, impatient, lengths, hq, hk, d, max_len):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(4)
    t = sum(lengths)
    q, k, v = torch.randn(t, hq + 2 * hk, d, generator=gen, device="cuda").bfloat16().split([hq, hk, hk], 1)
    cu = i32([0] + list(np.cumsum(lengths)))
    prompts = serve.PromptAttention()
    want, lse = torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(t, hq, device="cuda")
    out, lse2 = torch.empty_like(want), torch.empty_like(lse)
    prompts.attention(q, k, v, want, cu, max_len=max_len, lse=lse)
    assert prompts.status() == 0
    tok = (hq + 2 * hk) * d
    args = serve._PROMPT.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse2.data_ptr(), cu.data_ptr(),
                              prompts._workspace.data_ptr(), tok, d, tok, d, tok, d, hq * d, d, t, d ** -0.5, len(lengths), hq, hk, d,
                              0, max_len, 1, 0)
    impatient.rra_prompt_attention.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        flush.zero_()
        assert impatient.rra_prompt_attention(args, torch.cuda.current_stream().cuda_stream) == 0
        status = prompts.status()
        head = prompts._workspace[:4096].view(torch.int32)
        assert status == 5 and (head[1:] == 0).all()
        prompts.reset()
        prompts.attention(q, k, v, out, cu, max_len=max_len, lse=lse2)
        assert prompts.status() == 0 and torch.equal(out, want) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d", [64, 128])
def test_after_a_wait_ran_out_the_next_call_over_the_8_bit_cache_is_right(serve, impatient, d):  # noqa: F811
    from test_kv8_gpu import plans

    hq, hk, ps, new, kv = 16, 2, 64, [40, 300, 7, 0] + [1] * 20, [5000, 9000, 300, 10] + [4000] * 20
    held = [-(-n // ps) for n in kv]
    cache = serve.KvCache8(torch.zeros(sum(held), serve.kv8_page_bytes(ps, hk, d), dtype=torch.uint8, device="cuda"), ps, hk, d)
    table, used = torch.full((len(kv), max(held)), -1, dtype=torch.int32, device="cuda"), 0
    for b, n in enumerate(held):
        table[b, :n] = torch.arange(used, used + n, device="cuda")
        used += n
    gen = torch.Generator(device="cuda").manual_seed(4)
    slots = torch.arange(used * ps, device="cuda")
    cache.append(*(torch.randn(len(slots), hk, d, generator=gen, device="cuda") for _ in range(2)), slots)
    q = torch.randn(sum(new), hq, d, generator=gen, device="cuda").bfloat16()
    cu, kv_d = i32([0] + list(np.cumsum(new))), i32(kv)
    impatient.rra_kv8_attention.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    flush, ran_out = torch.empty(1 << 28, dtype=torch.uint8, device="cuda"), 0
    for max_q, max_kv in plans(cache, hq, len(new)).values():
        want, lse = torch.empty_like(q), torch.empty(q.shape[0], hq, device="cuda")
        out, lse2 = torch.empty_like(want), torch.empty_like(lse)
        cache.attention(q, want, cu, kv_d, table, max_q=max_q, max_kv=max_kv, lse=lse)
        assert cache.status() == 0
        flush.zero_()
        args = arguments(serve, cache, q, out, lse2, cu, kv_d, table, max_q, max_kv)
        assert impatient.rra_kv8_attention(args, torch.cuda.current_stream().cuda_stream) == 0
        ran_out += cache.status() == 5
        assert (cache._workspace[:4096].view(torch.int32)[1:] == 0).all()
        cache.reset()
        cache.attention(q, out, cu, kv_d, table, max_q=max_q, max_kv=max_kv, lse=lse2)
        assert cache.status() == 0 and torch.equal(out, want) and torch.equal(lse, lse2)
    assert ran_out >= 5


def test_two_prompts_objects_on_two_streams(serve):
    """Calls with workspaces of their own may run at the same time."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = torch.randn(3000, 16, 128, generator=gen, device="cuda").bfloat16().split([8, 4, 4], 1)
    cu = i32([0, 2500, 3000])
    a, b = serve.PromptAttention(), serve.PromptAttention()
    want = torch.empty(3000, 8, 128, dtype=torch.bfloat16, device="cuda")
    a.attention(q, k, v, want, cu, max_len=2500)
    outs = [torch.zeros_like(want) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, obj, out in zip(streams, (a, b), outs):
            obj.attention(q, k, v, out, cu, max_len=2500, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs) and a.status() == 0 and b.status() == 0


def test_kernels_that_need_tensor_memory_back_to_back(serve):
    """A grid may be on its way while the one before it ends, on the same SM and with the same tensor memory to share."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    ps, hq, hk, d, n = 64, 8, 4, 64, 1500
    q, k, v = torch.randn(n, hq + 2 * hk, d, generator=gen, device="cuda").bfloat16().split([hq, hk, hk], 1)
    pages = -(-n // ps)
    caches = [serve.KvCache(torch.zeros(pages, serve.kv_page_bytes(ps, hk, d), dtype=torch.uint8, device="cuda"), ps, hk, d),
              serve.KvCache8(torch.zeros(pages, serve.kv8_page_bytes(ps, hk, d), dtype=torch.uint8, device="cuda"), ps, hk, d)]
    table, cu, kv = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1), i32([0, n]), i32([n])
    for cache in caches:
        cache.append(k, v, torch.arange(n, device="cuda"))
    prompts = serve.PromptAttention()
    assert [prompts.plan_kernel(hq, hk, 1, max_len=m, tokens=n, head_dim=d) for m in (1, 10 ** 6)] == ["prompt_attention_kernel<128 rows>", "prompt_attention_kernel<256 rows>"]

    def calls(out):
        prompts.attention(q, k, v, out[0], cu, max_len=1)
        prompts.attention(q, k, v, out[1], cu, max_len=10 ** 6)
        for o, cache in zip(out[2:], caches):
            cache.attention(q, o, cu, kv, table, max_q=n, max_kv=n)

    want = [torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    calls(want)
    got = [torch.zeros_like(w) for w in want]
    for _ in range(50):
        calls(got)
    assert prompts.status() == 0 and all(c.status() == 0 for c in caches) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_tensors_of_another_kind_are_refused(serve):
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16, device="cuda")
    cu, prompts = i32([0, 4]), serve.PromptAttention()
    good = dict(q=q, k=q[:, :2], v=q[:, :2], out=q.clone(), cu=cu)

    def refused(error, **change):
        a = dict(good, **change)
        with pytest.raises(error):
            prompts.attention(a["q"], a["k"], a["v"], a["out"], a["cu"], max_len=4, lse=change.get("lse"))

    refused(TypeError, q=q.float())
    refused(ValueError, k=q[:, :2].half())
    refused(ValueError, k=q[:, :3])
    refused(ValueError, k=q[:2, :2])
    refused(ValueError, v=q[:, :1])
    refused(ValueError, out=q[:, :, ::2])
    refused(ValueError, out=q.cpu())
    refused(ValueError, cu=cu.long())
    refused(ValueError, lse=torch.zeros(4, 3, device="cuda"))
    for bad in (torch.zeros(4, 4, 132, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 4, 60, dtype=torch.bfloat16, device="cuda")):
        from latency_barrier_free_gb300 import rra
        with pytest.raises(rra.RraError):
            prompts.attention(bad, bad, bad, bad.clone(), cu, max_len=4)
    with pytest.raises(OverflowError):
        prompts.attention(q, good["k"], good["v"], good["out"], cu, max_len=2 ** 40)
    prompts.attention(q[:0], q[:0, :2], q[:0, :2], q[:0], i32([0]), max_len=0)
    prompts.attention(q, q[:, :2], q[:, :2], good["out"], i32([0]), max_len=4)
    assert prompts.status() == 0


def test_the_largest_batches(serve):
    """As many requests as a call takes, with and without tokens."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    lengths = [(b * 7) % 5 for b in range(4096)]
    t = sum(lengths)
    q, k, v = torch.randn(t, 6, 64, generator=gen, device="cuda").bfloat16().split([4, 1, 1], 1)
    out, prompts = torch.empty(t, 4, 64, dtype=torch.bfloat16, device="cuda"), serve.PromptAttention()
    cu = np.concatenate([[0], np.cumsum(lengths)])
    prompts.attention(q, k, v, out, i32(list(cu)), max_len=4)
    for b in (0, 3, 2048, 4095):
        for i in range(cu[b], cu[b + 1]):
            s = torch.einsum("hd,kd->hk", q[i].double(), k[cu[b]:i + 1, 0].double()) / 8
            want = s.softmax(-1) @ v[cu[b]:i + 1, 0].double()
            assert ((out[i].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -7 * v[cu[b]:i + 1].abs().max()).all()
    assert prompts.status() == 0
