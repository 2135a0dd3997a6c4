"""Refusals of the 8-bit cache and the shared pages (host checks, no GPU needed), the sizes of their argument
structures, and the references of their tests."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import more_serve_ref as more
from latency_barrier_free_gb300 import rra
from test_serve_cpu import FAKE, ROOT, fields, refused, serve  # noqa: F401

torch = pytest.importorskip("torch")

STRUCTS = {"rra_pages_fork_args_t": "_FORK", "rra_pages_release_args_t": "_RELEASE", "rra_pages_compact_args_t": "_COMPACT",
           "rra_pages_copy_args_t": "_COPY", "rra_prompt_attention_args_t": "_PROMPT"}


def test_structures_have_the_headers_sizes(serve, tmp_path):  # noqa: F811
    c = tmp_path / "sizes.c"
    c.write_text('#include <stdio.h>\n#include "rra_serve.h"\nint main(void) {\n%s return 0; }\n'
                 % "\n".join('printf("%%zu\\n", sizeof(%s));' % n for n in STRUCTS))
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(exe)], check=True)
    sizes = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert sizes == [getattr(serve, n).size for n in STRUCTS.values()]


def test_page_bytes(serve):  # noqa: F811
    assert serve.kv8_page_bytes(64, 8, 128) == 4 * 8 * 4112 and serve.kv8_page_bytes(16, 1, 64) == 2064
    for bad in ((0, 1, 64), (8, 1, 64), (24, 1, 64), (8192, 1, 64), (16, 0, 64), (16, 1, 96), (16, 1, 256)):
        with pytest.raises(rra.RraError) as e:
            serve.kv8_page_bytes(*bad)
        assert e.value.status == rra.ERR_INVALID_ARG


def test_cache_refusals(serve):  # noqa: F811
    names = fields("rra_kv_tokens_args_t")
    good = [FAKE, 100, 16, 8, 128, 0] + [FAKE] * 3 + [1024, 128] * 2 + [5, 1, 0]
    for fn in ("rra_kv8_append", "rra_kv8_read"):
        refused(serve, fn, serve._TOKENS, good, [
            ("pages", 0), ("pages", FAKE + 8), ("num_pages", -1), ("page_tokens", 20), ("kv_heads", 0), ("head_dim", 32),
            ("k", 0), ("v", 0), ("k", FAKE + 4), ("slots", 0), ("k_token_stride", 0), ("v_head_stride", 100),
            ("k_head_stride", 132), ("tokens", -1), ("tokens", 2 ** 31), ("dtype", 2), ("dtype", -1)], names)
        assert serve._lib()[fn](serve._TOKENS.pack(*(good[:-3] + [0, 1, 0])), 0) == rra.OK
    names = fields("rra_kv_attention_args_t")
    good = [FAKE, 100, 16, 2, 128, 0] + [FAKE] * 7 + [1024, 128] * 2 + [8, 5, 0.1, 3, 8, 8, 1, 100, 1, 0, 0]
    refused(serve, "rra_kv8_attention", serve._ATTN, good, [
        ("pages", 0), ("head_dim", 96), ("q", 0), ("out", 0), ("cu_q", 0), ("kv_len", 0), ("block_table", 0), ("workspace", 0),
        ("workspace", FAKE + 16), ("q", FAKE + 2), ("q_token_stride", 0), ("out_head_stride", 4), ("table_stride", 7),
        ("tokens", -1), ("scale", float("inf")), ("scale", float("nan")), ("requests", 4097), ("q_heads", 7), ("max_q", -1),
        ("window", -1)], names)
    name = ctypes.c_char_p()
    assert serve._lib().rra_kv8_attention_plan(serve._ATTN.pack(*good), ctypes.byref(name)) == rra.OK
    assert name.value.decode().startswith("kv_attention")
    assert serve._lib().rra_kv8_attention_plan(serve._ATTN.pack(*good), None) == rra.ERR_INVALID_ARG


def test_prompt_refusals(serve):  # noqa: F811
    names = fields("rra_prompt_attention_args_t")
    good = [FAKE] * 7 + [1024, 128, 512, 128, 512, 128, 1024, 128, 100, 0.1, 3, 8, 4, 128, 0, 60, 1, 0]
    assert len(names) == len(good)
    refused(serve, "rra_prompt_attention", serve._PROMPT, good, [
        ("q", 0), ("k", 0), ("v", 0), ("out", 0), ("cu", 0), ("workspace", 0), ("workspace", FAKE + 16), ("q", FAKE + 8),
        ("k", FAKE + 2), ("q_token_stride", 0), ("k_head_stride", 100), ("v_token_stride", 516), ("out_head_stride", 4),
        ("q_token_stride", 2 ** 39), ("tokens", -1), ("tokens", 2 ** 30), ("tokens", 2 ** 27), ("scale", float("inf")),
        ("scale", float("nan")), ("scale", 3e38), ("requests", -1), ("requests", 4097), ("q_heads", 0), ("q_heads", 7),
        ("kv_heads", 0), ("head_dim", 0), ("head_dim", 100), ("head_dim", 136), ("half", 2), ("half", -1), ("max_len", -1),
        ("window", -1)], names)
    for name in ("requests", "tokens"):  # nothing to do
        args = list(good)
        args[names.index(name)] = 0
        assert serve._lib().rra_prompt_attention(serve._PROMPT.pack(*args), 0) == rra.OK
    name = ctypes.c_char_p()
    plan = serve._lib().rra_prompt_attention_plan
    for longest, rows in ((0, 128), (64, 128), (100000, 256), (2 ** 31 - 1, 256)):
        args = list(good)
        args[names.index("max_len")] = longest
        assert plan(serve._PROMPT.pack(*args), ctypes.byref(name)) == rra.OK
        assert name.value.decode() == "prompt_attention_kernel<%d rows>" % rows
    assert plan(serve._PROMPT.pack(*good), None) == rra.ERR_INVALID_ARG
    assert serve._lib().rra_prompt_attention_workspace_bytes() > 4096


def test_fork_refusals(serve):  # noqa: F811
    names = fields("rra_pages_fork_args_t")
    good = [FAKE] * 13 + [8, 4, 3, 8, 16, 100, 0]
    assert len(names) == len(good)
    refused(serve, "rra_pages_fork", serve._FORK, good, [(n, 0) for n in names[:13]] + [
        ("table_stride", 7), ("requests", -1), ("requests", 4097), ("forks", -1), ("forks", 4097), ("table_pages", -1),
        ("page_tokens", 0), ("num_pages", -1), ("num_pages", 2 ** 24 + 1), ("num_pages", 2 ** 31 - 1), ("reserved", 1)], names)


def test_release_refusals(serve):  # noqa: F811
    names = fields("rra_pages_release_args_t")
    good = [FAKE] * 9 + [8, 4, 8, 16, 100]
    assert len(names) == len(good)
    refused(serve, "rra_pages_release", serve._RELEASE, good, [(n, 0) for n in names[:9]] + [
        ("table_stride", 7), ("requests", -1), ("requests", 4097), ("table_pages", -1), ("page_tokens", 0), ("num_pages", -1),
        ("num_pages", 2 ** 24 + 1), ("num_pages", 2 ** 31 - 1)], names)


def test_compact_refusals(serve):  # noqa: F811
    names = fields("rra_pages_compact_args_t")
    good = [FAKE] * 13 + [8, 8, 4, 8, 16, 100, 5, 0]
    assert len(names) == len(good)
    refused(serve, "rra_pages_compact", serve._COMPACT, good, [(n, 0) for n in names[:13]] + [
        ("table_stride", 7), ("table_out_stride", 7), ("table_out_stride", 9), ("requests", -1), ("requests", 4097),
        ("table_pages", -1), ("page_tokens", 0), ("num_pages", -1), ("num_pages", 2 ** 24 + 1), ("num_pages", 2 ** 31 - 1), ("max_moves", -1),
        ("reserved", 1)], names)


def test_copy_refusals(serve):  # noqa: F811
    names = fields("rra_pages_copy_args_t")
    good = [FAKE] * 4 + [10, 10, 1152, 3, 0]
    assert len(names) == len(good)
    refused(serve, "rra_pages_copy", serve._COPY, good, [(n, 0) for n in names[:4]] + [
        ("from_pages", FAKE + 8), ("to_pages", FAKE + 4), ("from_num", -1), ("to_num", -1), ("page_bytes", 0), ("page_bytes", 24),
        ("page_bytes", 2 ** 41), ("count", -1), ("reserved", 1)], names)
    for name in ("count", "from_num", "to_num"):  # nothing to do
        args = list(good)
        args[names.index(name)] = 0
        assert serve._lib().rra_pages_copy(serve._COPY.pack(*args), 0) == rra.OK


def test_tensors_that_are_not_on_a_gpu_are_refused(serve):  # noqa: F811
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        serve.pages_fork(i, i, i, i.view(4, 1), i, i, i, 16, kv_len=i, shared_out=i, copy_from=i, copy_to=i, free_left=i,
                         pages_short=i)
    with pytest.raises(ValueError):
        serve.pages_release(i, i, i.view(4, 1), i, i, i, 16, kv_len=i, shared_out=i, free_left=i)
    with pytest.raises(ValueError):
        serve.pages_compact(i, i.view(4, 1), i, i, i, 16, table_out=i.view(4, 1), free_out=i, shared_out=i, free_left=i, moved=i,
                            move_from=i, move_to=i, move_count=i)
    with pytest.raises(ValueError):
        serve.KvCache8(torch.zeros(4, serve.kv8_page_bytes(16, 1, 64), dtype=torch.uint8), 16, 1, 64)


def test_references_agree_with_themselves():
    """Rounding against a table of all codes, the layout, and a small write by hand."""
    every = np.arange(127)
    assert np.array_equal(more.e4m3(more.values(every)), every) and more.values(126) == 448 and more.values(1) == 2.0 ** -9
    grid = more.values(every)
    for low, high, code in zip(grid, grid[1:], every):
        mid = (low + high) / 2
        assert more.e4m3(mid) == code + code % 2 and more.e4m3(mid * (1 + 1e-9)) == code + 1 and more.e4m3(mid * (1 - 1e-9)) == code
    assert more.e4m3(1e9) == 126 and more.e4m3(-np.inf) == 254
    if hasattr(torch, "float8_e4m3fn"):
        x = np.random.default_rng(0).standard_normal(4096) * 40
        t = torch.from_numpy(x).float()
        assert np.array_equal(more.e4m3(t.double().numpy()), t.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    for d in (64, 128):
        assert sorted(more.at(d).flatten()) == list(range(16 * d))
    assert [more.exponent(x) for x in ([448.0], [448.5], [0.0], [1e30], [np.inf, 2.0])] == [0, 1, -32, 32, -7]
    pages = np.zeros((1, 1 * 2064), np.uint8)
    x = np.full((2, 1, 64), 3.0, np.float32)
    x[1] = 500.0
    more.append8(pages, 16, 1, 64, x, -x, [0, 1])
    k, v = more.read8(pages, 16, 1, 64, [0, 1, 2, -1])
    assert k[0, 0, 0] == 3.0 and k[1, 0, 5] == 512.0 and v[1, 0, 5] == -512.0 and (k[2:] == 0).all()


def test_reference_pages_by_hand():
    table, shared = np.array([[4, 2], [-1, -1]], np.int32), np.zeros(6, np.int32)
    kv, frm, to, left, short = more.fork([20, 0], [0], [1], table, np.array([0, 1, 3, 5, 0, 0]), 4, shared, 16)
    assert kv == [20, 20] and (frm, to, left, short) == ([2], [5], 3, 0) and table[1].tolist() == [4, 5] and shared[4] == 1
    free = np.array([0, 1, 3, 0, 0, 0])
    kv, left = more.release([20, 20], [-1, 1], table, free, 3, shared, 16)
    assert kv == [0, 20] and left == 4 and free[3] == 2 and shared.sum() == 0
    t, f, left, s, moved, moves = more.compact([0, 20], table, free, 4, shared, 16, 9)
    assert moves == [(5, 0), (4, 1)] and t[1].tolist() == [1, 0] and f[:4].tolist() == [5, 4, 3, 2] and moved[5] == 0
