"""Refusals of the decode-step operators (host checks, no GPU needed), the
sizes of their argument structures, and the references of their tests."""
import ctypes
import os
import re
import struct
import subprocess

import numpy as np
import pytest

import serve_ref as ref
from latency_barrier_free_gb300 import build_ext, rra

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def serve():
    build_ext.build()
    from latency_barrier_free_gb300 import serve

    return serve


def test_page_bytes_and_workspace(serve):
    lib = serve._lib()
    assert serve.kv_page_bytes(64, 8, 128) == 64 * 8 * 144
    assert serve.kv_page_bytes(16, 1, 64) == 16 * 72
    for bad in ((0, 1, 64), (8, 1, 64), (24, 1, 64), (8192, 1, 64), (16, 0, 64), (16, 1, 96), (16, 1, 256)):
        with pytest.raises(rra.RraError) as e:
            serve.kv_page_bytes(*bad)
        assert e.value.status == rra.ERR_INVALID_ARG
    assert lib.rra_kv_attention_workspace_bytes(128) > 4096 and lib.rra_kv_attention_workspace_bytes(32) == 0


def test_structures_have_the_headers_sizes(serve, tmp_path):
    c = tmp_path / "sizes.c"
    c.write_text('#include <stdio.h>\n#include "rra_serve.h"\nint main(void) { printf("%zu %zu %zu %zu\\n", '
                 "sizeof(rra_slot_map_args_t), sizeof(rra_qk_norm_rope_args_t), sizeof(rra_kv_tokens_args_t), "
                 "sizeof(rra_kv_attention_args_t)); return 0; }\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(exe)], check=True)
    sizes = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert sizes == [serve._SLOTS.size, serve._ROPE.size, serve._TOKENS.size, serve._ATTN.size]


FAKE = 1 << 20  # an aligned address; a refused call never touches it


def refused(serve, fn, fmt, good, changes, names):
    """`good` with any of `changes` is refused before anything is launched."""
    f = getattr(serve._lib(), fn)
    for name, value in changes:
        args = list(good)
        args[names.index(name)] = value
        assert f(fmt.pack(*args), 0) == rra.ERR_INVALID_ARG, (fn, name, value)
    assert f(None, 0) == rra.ERR_INVALID_ARG


def fields(struct_name, inner=None):
    """Field names of a structure of rra_serve.h, in order."""
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "rra_serve.h")).read(), flags=re.S)
    body = [m.group(1) for m in re.finditer(r"typedef struct \{([^}]*)\} (\w+);", text) if m.group(2) == struct_name][0]
    out = []
    for line in body.split(";"):
        line = line.strip()
        if not line:
            continue
        if line.startswith("rra_kv_cache_t"):
            out += fields("rra_kv_cache_t")
            continue
        first, *rest = line.split(",")
        out += [re.findall(r"\w+", x)[-1] for x in [first] + rest]
    return out


def test_slot_map_refusals(serve):
    names = fields("rra_slot_map_args_t")
    good = [FAKE] * 11 + [8, 64, 4, 8, 16, 100]
    assert len(names) == len(good)
    refused(serve, "rra_slot_map", serve._SLOTS, good, [
        ("requests", -1), ("requests", 4097), ("tokens", -1), ("tokens", 2 ** 31), ("page_tokens", 0), ("num_pages", -1),
        ("table_pages", -1), ("table_stride", 7), ("seq_len", 0), ("new_len", 0), ("block_table", 0), ("free_pages", 0),
        ("free_count", 0), ("kv_len", 0), ("cu_new", 0), ("slots", 0), ("positions", 0), ("free_left", 0),
        ("pages_short", 0)], names)


def test_qk_norm_rope_refusals(serve):
    names = fields("rra_qk_norm_rope_args_t")
    good = [FAKE] * 9 + [1024, 128] * 4 + [5, 100, 1e-6, 8, 8, 128, 128, 0, 1]
    assert len(names) == len(good)
    refused(serve, "rra_qk_norm_rope", serve._ROPE, good, [
        ("q", 0), ("k", 0), ("q_out", 0), ("k_out", 0), ("q", FAKE + 2), ("k_out", FAKE + 8), ("q_weight", FAKE + 4),
        ("cos", 0), ("sin", 0), ("positions", 0), ("cos", FAKE + 4), ("q_token_stride", 0), ("q_token_stride", 1025),
        ("q_head_stride", 127), ("q_head_stride", 64), ("k_out_head_stride", 129), ("tokens", -1), ("eps", -1.0),
        ("eps", float("nan")), ("q_heads", -1), ("head_dim", 120), ("head_dim", 272), ("head_dim", 0), ("rot", 24),
        ("rot", 144), ("rot", -16), ("max_position", -1), ("dtype", 2), ("dtype", 7)], names)
    zero = list(good)
    zero[names.index("tokens")] = 0
    assert serve._lib().rra_qk_norm_rope(serve._ROPE.pack(*zero), 0) == rra.OK


def test_append_and_read_refusals(serve):
    names = fields("rra_kv_tokens_args_t")
    good = [FAKE, 100, 16, 8, 128, 0] + [FAKE] * 3 + [1024, 128] * 2 + [5, 1, 0]
    assert len(names) == len(good)
    for fn in ("rra_kv_append", "rra_kv_read"):
        refused(serve, fn, serve._TOKENS, good, [
            ("pages", 0), ("pages", FAKE + 8), ("num_pages", -1), ("page_tokens", 20), ("kv_heads", 0), ("head_dim", 32),
            ("k", 0), ("v", 0), ("k", FAKE + 4), ("slots", 0), ("k_token_stride", 0), ("v_head_stride", 100),
            ("k_head_stride", 132), ("tokens", -1), ("dtype", 2), ("dtype", -1)], names)
        assert serve._lib()[fn](serve._TOKENS.pack(*(good[:-3] + [0, 1, 0])), 0) == rra.OK


def test_attention_refusals(serve):
    names = fields("rra_kv_attention_args_t")
    good = [FAKE, 100, 16, 2, 128, 0] + [FAKE] * 7 + [1024, 128] * 2 + [8, 5, 0.1, 3, 8, 8, 1, 100, 1, 0, 0]
    assert len(names) == len(good)
    refused(serve, "rra_kv_attention", serve._ATTN, good, [
        ("pages", 0), ("head_dim", 96), ("q", 0), ("out", 0), ("cu_q", 0), ("kv_len", 0), ("block_table", 0),
        ("workspace", 0), ("workspace", FAKE + 16), ("q", FAKE + 2), ("q_token_stride", 0), ("out_head_stride", 4),
        ("q_head_stride", 130), ("table_stride", 7), ("tokens", -1), ("tokens", 2 ** 31), ("scale", float("inf")),
        ("scale", float("nan")), ("requests", -1), ("requests", 4097), ("table_pages", -1), ("q_heads", 0), ("q_heads", 7),
        ("max_q", -1), ("max_kv", -1), ("window", -1)], names)
    name = ctypes.c_char_p()
    assert serve._lib().rra_kv_attention_plan(serve._ATTN.pack(*good), ctypes.byref(name)) == rra.OK
    assert name.value.decode().startswith("kv_attention")
    assert serve._lib().rra_kv_attention_plan(serve._ATTN.pack(*good), None) == rra.ERR_INVALID_ARG
    none = list(good)
    none[names.index("requests")] = 0
    assert serve._lib().rra_kv_attention(serve._ATTN.pack(*none), 0) == rra.OK


def test_tensors_that_are_not_on_a_gpu_are_refused(serve):
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        serve.slot_map(i, i, i.view(4, 1), i, i, 16, kv_len=i, cu_new=i, slots=i.long(), positions=i, free_left=i,
                       pages_short=i)
    with pytest.raises(ValueError):
        serve.KvCache(torch.zeros(4, serve.kv_page_bytes(16, 1, 64), dtype=torch.uint8), 16, 1, 64)
    x = torch.zeros(2, 2, 64)
    with pytest.raises(ValueError):
        serve.qk_norm_rope(x, x, None, None, None, None, None, x, x)


def test_references_agree_with_themselves():
    """The byte layout is a bijection, and writing then reading pages returns the quantised values."""
    for d in (64, 128):
        at, shift = ref.byte_and_shift(d)
        assert len(set(zip(at.tolist(), shift.tolist()))) == d and at.max() == d // 2 - 1
    rng = np.random.default_rng(0)
    pages = np.full((3, 2 * 18 * 64 * 2), 0xA5, np.uint8)
    x = rng.standard_normal((20, 2, 64)).astype(np.float32)
    slots = rng.permutation(96)[:20]
    ref.write_pages(pages, 32, 2, 64, x, 2 * x, slots)
    k, v = ref.read_pages(pages, 32, 2, 64, slots)
    assert np.array_equal(k, ref.dequantise(*ref.quantise(x))) and np.array_equal(v, 2 * k)
    assert np.abs(k - x).max() < 0.5 and struct.calcsize("P") == 8


def test_reference_slot_map_by_hand():
    table, free = np.array([[5, 6, -1], [2, -1, -1]], np.int32), np.array([9, 8, 0, 0], np.int32)
    kv, cu, slots, pos, top, short = ref.slot_map([4, 2], [-1, 3], table, np.r_[free, np.zeros(6, np.int32)], 2, 2, 5)
    # 5 and 6 go back on the stack; request 1 (tokens 2, 3, 4) gets 6, then 5
    assert kv == [0, 5] and cu == [0, 0, 3] and slots == [12, 13, 10, -1, -1] and pos == [2, 3, 4, 0, 0] and (top, short) == (2, 0)
