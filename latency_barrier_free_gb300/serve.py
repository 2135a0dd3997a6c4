"""Python binding of the serving operators (include/rra_serve.h).

Page bookkeeping, head norms with position rotation, a key/value cache held in
4 or 8 bits, and the attention over it: what a tensor-parallel rank runs around its
AllReduces; attention of whole prompts, and pages that several requests share.  As
in rra.py this is argument checking and marshalling only (in _serve.so,
csrc/serve_bind.cpp); every call enqueues one kernel of librra.so on the
current stream (or `stream`), and there is no fallback.  Tensors are on the current
GPU; those of another one are refused.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os
import struct

import torch

from . import rra

NATIVE_PATH = os.path.join(rra.HERE, "_serve.so")

_SLOTS = struct.Struct("11P2q4i")
_ROPE = struct.Struct("9P10qd6i")
_TOKENS = struct.Struct("Pq4i3P5q2i")
_ATTN = struct.Struct("Pq4i7P6qd8i")
_CACHE = struct.Struct("Pq4i")
_PROMPT = struct.Struct("7P9qd8i")
_FORK = struct.Struct("13Pq6i")
_RELEASE = struct.Struct("9Pq4i")
_COMPACT = struct.Struct("13P2q6i")
_COPY = struct.Struct("4P3q2i")

_WORKSPACE_HEAD = 4096  # bytes of the workspace that a call expects to be zero

_fns = None


def _lib():
    """The operators' entry points (loads the library on first use)."""
    global _fns
    if _fns is None:
        lib = rra.load()
        vp = ctypes.c_void_p
        sig = {"rra_slot_map": [vp, vp], "rra_qk_norm_rope": [vp, vp], "rra_kv_append": [vp, vp],
               "rra_kv_read": [vp, vp], "rra_kv_attention": [vp, vp],
               "rra_kv_attention_plan": [vp, ctypes.POINTER(ctypes.c_char_p)],
               "rra_kv8_append": [vp, vp], "rra_kv8_read": [vp, vp], "rra_kv8_attention": [vp, vp],
               "rra_kv8_attention_plan": [vp, ctypes.POINTER(ctypes.c_char_p)], "rra_prompt_attention": [vp, vp],
               "rra_prompt_attention_plan": [vp, ctypes.POINTER(ctypes.c_char_p)], "rra_pages_fork": [vp, vp],
               "rra_pages_release": [vp, vp], "rra_pages_compact": [vp, vp], "rra_pages_copy": [vp, vp]}
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, ctypes.c_int
        for fn in (lib.rra_kv_page_bytes, lib.rra_kv8_page_bytes):
            fn.argtypes, fn.restype = [ctypes.c_int] * 3, ctypes.c_size_t
        lib.rra_kv_attention_workspace_bytes.argtypes = [ctypes.c_int]
        lib.rra_kv_attention_workspace_bytes.restype = ctypes.c_size_t
        lib.rra_prompt_attention_workspace_bytes.argtypes = []
        lib.rra_prompt_attention_workspace_bytes.restype = ctypes.c_size_t
        _fns = lib
    return _fns


class _Native:
    """_serve.so, loaded on first use: until then any of its functions loads it."""

    def __getattr__(self, name):
        global _native
        _lib()
        if not os.path.exists(NATIVE_PATH):
            raise RuntimeError("_serve.so not found at %s; run latency_barrier_free_gb300.build_ext.build()" % NATIVE_PATH)
        loader = importlib.machinery.ExtensionFileLoader("_serve", NATIVE_PATH)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_serve", loader))
        loader.exec_module(module)
        module.init(rra.LIB_PATH)
        _native = module
        return getattr(module, name)


_native = _Native()


def _device(t):
    d = t.get_device()
    if d < 0 or t.dim() < 1:
        raise ValueError("expected CUDA tensors")
    return d


def slot_map(seq_len, new_len, block_table, free_pages, free_count, page_tokens, *, kv_len, cu_new, slots, positions,
             free_left, pages_short, stream=None) -> None:
    """One step of the paged cache's bookkeeping (rra_slot_map): requests with
    new_len[b] < 0 give their pages back, the others get the pages their new
    tokens need; writes kv_len, cu_new, slots, positions, free_left, pages_short
    and the new entries of block_table.  slots.numel() is the fixed number of
    tokens of the step.  Lengths, tables and pages are int32, slots int64."""
    st = _native.slot_map(seq_len, new_len, block_table, free_pages, free_count, page_tokens, kv_len, cu_new, slots, positions,
                          free_left, pages_short, stream)
    if st:
        raise rra.RraError(st, "rra_slot_map")


def qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, q_out, k_out, *, eps: float = 1e-6,
                 interleaved: bool = False, stream=None) -> None:
    """Norms of queries and keys for each head and the position rotation, in one
    pass (rra_qk_norm_rope).  q [tokens, q_heads, d] and k [tokens, k_heads, d]
    may be views of a packed projection; q_out and k_out may be q and k.  A
    weight of None leaves out that tensor's norm.  cos and sin are float32
    [max_position, rot/2], or None for no rotation; `interleaved` pairs
    neighbouring channels instead of halves."""
    st = _native.qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, q_out, k_out, eps, interleaved, stream)
    if st:
        raise rra.RraError(st, "rra_qk_norm_rope")


def kv_page_bytes(page_tokens: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of one page of the 4-bit cache."""
    n = _lib().rra_kv_page_bytes(page_tokens, kv_heads, head_dim)
    if n == 0:
        raise rra.RraError(rra.ERR_INVALID_ARG, "rra_kv_page_bytes")
    return n


def kv8_page_bytes(page_tokens: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of one page of the 8-bit cache."""
    n = _lib().rra_kv8_page_bytes(page_tokens, kv_heads, head_dim)
    if n == 0:
        raise rra.RraError(rra.ERR_INVALID_ARG, "rra_kv8_page_bytes")
    return n


def pages_fork(seq_len, source, target, block_table, free_pages, free_count, shared, page_tokens, *, kv_len, shared_out,
               copy_from, copy_to, free_left, pages_short, stream=None) -> None:
    """Requests that continue others (rra_pages_fork): row target[i] becomes a copy
    of row source[i], whose whole pages both share from then on (shared counts a
    page's holders beyond the first); the last one, if it is not full, gets a page
    of its own, and copy_from[i], copy_to[i] say what to copy: give them to copy() of
    the cache of every layer.  All int32; kv_len may be seq_len, shared_out shared,
    free_left free_count."""
    st = _native.pages_fork(seq_len, source, target, block_table, free_pages, free_count, shared, page_tokens, kv_len, shared_out,
                            copy_from, copy_to, free_left, pages_short, stream)
    if st:
        raise rra.RraError(st, "rra_pages_fork")


def pages_release(seq_len, new_len, block_table, free_pages, free_count, shared, page_tokens, *, kv_len, shared_out, free_left,
                  stream=None) -> None:
    """Requests with new_len[b] < 0 end (rra_pages_release): their pages go back on
    the stack once nobody else holds them, and their kv_len is 0, so that slot_map
    with the same new_len returns nothing for them again.  kv_len may be seq_len,
    shared_out shared, free_left free_count."""
    st = _native.pages_release(seq_len, new_len, block_table, free_pages, free_count, shared, page_tokens, kv_len, shared_out,
                               free_left, stream)
    if st:
        raise rra.RraError(st, "rra_pages_release")


def pages_compact(seq_len, block_table, free_pages, free_count, shared, page_tokens, *, table_out, free_out, shared_out, free_left,
                  moved, move_from, move_to, move_count, stream=None) -> None:
    """Moves the highest pages in use to the lowest free ones, at most
    move_from.numel() (rra_pages_compact): new tables, stack and counts, moved[p] the
    new number of page p (-1: it was free), and the moves (-1 behind the last), which
    copy() of the cache of every layer carries out.  table_out may be block_table,
    free_out free_pages, free_left free_count, shared_out shared."""
    st = _native.pages_compact(seq_len, block_table, free_pages, free_count, shared, page_tokens, table_out, free_out, shared_out,
                               free_left, moved, move_from, move_to, move_count, stream)
    if st:
        raise rra.RraError(st, "rra_pages_compact")


class _Workspace:
    """What an attention's calls need besides their tensors: memory, with a status word in front."""

    def _allocate(self, size: int, dev: int):
        self._dev = dev
        self._workspace = torch.empty(size, dtype=torch.uint8, device=torch.device("cuda", dev))
        self._workspace[:_WORKSPACE_HEAD].zero_()
        own = torch.cuda.current_stream(dev)
        if not torch.cuda.is_current_stream_capturing():
            own.synchronize()  # calls on other streams find the zeros
        self._home = own.cuda_stream

    def status(self) -> int:
        """Status word of the attention calls so far (0 is fine), whatever their
        stream; synchronises with the GPU."""
        torch.cuda.synchronize(self._dev)
        return int(self._workspace[:4].cpu().view(torch.int32).item())

    def reset(self) -> None:
        """Sets the status back to 0, in the order of the current stream: after a
        status that is not, attention() gives valid results from here on."""
        self._workspace[:_WORKSPACE_HEAD].zero_()


class PromptAttention(_Workspace):
    """Attention of whole prompts over their own keys and values.

    The object holds the attention's workspace, on the current GPU: its calls are
    ordered on one stream, any one.  It may go once they are enqueued, but for calls
    whose stream was given as a number, which it has to outlive, and for graphs that
    hold calls."""

    def __init__(self):
        self._allocate(_lib().rra_prompt_attention_workspace_bytes(), torch.cuda.current_device())

    def attention(self, q, k, v, out, cu, *, max_len: int, scale=None, causal: bool = True, window: int = 0, lse=None,
                  stream=None) -> None:
        """out = attention of q [tokens, q_heads, head_dim] over k and v [tokens,
        kv_heads, head_dim], all bfloat16 or all float16 (rra_prompt_attention): prompt
        b has the tokens cu[b]..cu[b+1] (int32) of all of them, each of which sees the
        prompt's tokens up to itself (all of them, unless `causal`), the last `window`
        of them if that is not 0.  max_len is what to plan for; scale defaults to
        1/sqrt(head_dim); scores are below 2^26.  lse: float32 [tokens, q_heads], optional.  Rows of out and lse
        after cu[-1], a step's padding, stay as they are."""
        st = _native.prompt_attention(self._dev, self._workspace, q, k, v, out, cu, max_len, scale, causal, window, lse, stream,
                                      self._home)
        if st:
            raise rra.RraError(st, "rra_prompt_attention")

    def plan_kernel(self, q_heads: int, kv_heads: int, requests: int, *, max_len: int, tokens=None, head_dim: int = 128,
                    causal: bool = True, window: int = 0) -> str:
        """Name of the kernel that attention() launches for so many requests of max_len
        tokens at most, and `tokens` rows (requests * max_len, if not given)."""
        some = self._workspace.data_ptr()  # planning reads no memory
        rows = requests * max_len if tokens is None else tokens
        args = _PROMPT.pack(some, some, some, some, 0, some, some, q_heads * 128, 128, kv_heads * 128, 128, kv_heads * 128, 128,
                            q_heads * 128, 128, rows, 1.0, requests, q_heads, kv_heads, head_dim, 0, max_len, int(causal), window)
        name = ctypes.c_char_p()
        st = _lib().rra_prompt_attention_plan(args, ctypes.byref(name))
        if st:
            raise rra.RraError(st, "rra_prompt_attention_plan")
        return name.value.decode()


class KvCache(_Workspace):
    """A paged key/value cache held in 4 bits, in memory of the caller.

    `pages` is a contiguous uint8 CUDA tensor of whole pages (kv_page_bytes()
    each; their layout stands in rra_serve.h); it needs no initialisation.  The
    object holds the attention's workspace, so its attention() calls are ordered
    on one stream, any one; append() and read() are not bound to it.  It may go
    once they are enqueued, but for calls whose stream was given as a number, which
    it has to outlive, and for graphs that hold calls."""

    _size = staticmethod(kv_page_bytes)
    _plan = "rra_kv_attention_plan"

    def __init__(self, pages, page_tokens: int, kv_heads: int, head_dim: int):
        lib = _lib()
        size = self._size(page_tokens, kv_heads, head_dim)
        dev = _device(pages)
        if pages.dtype is not torch.uint8 or not pages.is_contiguous() or pages.numel() % size:
            raise ValueError("pages must be a contiguous uint8 tensor of whole pages (%d bytes each)" % size)
        self.pages, self.page_bytes = pages, size
        self.page_tokens, self.kv_heads, self.head_dim = int(page_tokens), int(kv_heads), int(head_dim)
        self.num_pages = pages.numel() // size
        self._allocate(lib.rra_kv_attention_workspace_bytes(head_dim), dev)
        self._cache = _CACHE.pack(pages.data_ptr(), self.num_pages, self.page_tokens, self.kv_heads, self.head_dim, 0)
        self._scale = 1.0 / math.sqrt(head_dim)

    def append(self, k, v, slots, stream=None) -> None:
        """Write k and v [tokens, kv_heads, head_dim] to the slots (int64;
        negative: skipped)."""
        st = _native.kv_append(self._cache, self._dev, k, v, slots, stream)
        if st:
            raise rra.RraError(st, "rra_kv_append")

    def read(self, slots, k, v, stream=None) -> None:
        """k and v [tokens, kv_heads, head_dim] become the values that the slots hold."""
        st = _native.kv_read(self._cache, self._dev, k, v, slots, stream)
        if st:
            raise rra.RraError(st, "rra_kv_read")

    def attention(self, q, out, cu_q, kv_len, block_table, *, max_q: int, max_kv: int, scale=None, causal: bool = True,
                  window: int = 0, lse=None, stream=None) -> None:
        """out = attention of q [tokens, q_heads, head_dim] (bfloat16) over the
        cache (rra_kv_attention).  Request b has the queries cu_q[b]..cu_q[b+1]
        and the first kv_len[b] tokens of its row of block_table, its own
        included; max_q and max_kv are what to plan for.  scale defaults to
        1/sqrt(head_dim).  lse: float32 [tokens, q_heads], optional.  Rows of out
        and lse after cu_q[-1], a step's padding, stay as they are."""
        st = _native.kv_attention(self._cache, self._dev, self._workspace, q, out, cu_q, kv_len, block_table, max_q, max_kv,
                                  self._scale if scale is None else scale, causal, window, lse, stream, self._home)
        if st:
            raise rra.RraError(st, "rra_kv_attention")

    def plan_kernel(self, q_heads: int, requests: int, *, max_q: int, max_kv: int, window: int = 0) -> str:
        """Name of the kernel that attention() launches for so many query heads
        and requests and this window, planned for max_q and max_kv."""
        some = self._workspace.data_ptr()  # planning reads no memory
        d = self.head_dim
        args = _ATTN.pack(*_CACHE.unpack(self._cache), some, some, 0, some, some, some, some, q_heads * d, d, q_heads * d, d, 1,
                          requests, self._scale, requests, 1, q_heads, max_q, max_kv, 1, window, 0)
        name = ctypes.c_char_p()
        st = getattr(_lib(), self._plan)(args, ctypes.byref(name))
        if st:
            raise rra.RraError(st, self._plan)
        return name.value.decode()

    def copy(self, source, target, to=None, stream=None) -> None:
        """Page target[i] becomes a copy of page source[i] (rra_pages_copy; int32, pairs
        with a number outside the cache are skipped), of this cache or of `to`, a cache
        of the same kind.  Not ordered with other streams, like append()."""
        to = self if to is None else to
        if type(to) is not type(self) or (to.page_tokens, to.kv_heads, to.head_dim) != (self.page_tokens, self.kv_heads, self.head_dim):
            raise ValueError("pages are copied between caches of one kind, page size and heads")
        st = _native.pages_copy(self.pages, to.pages, self.page_bytes, source, target, stream)
        if st:
            raise rra.RraError(st, "rra_pages_copy")


class KvCache8(KvCache):
    """The same over a cache held in 8 bits: e4m3 codes, and an exponent for each
    block of 16 tokens and head (kv8_page_bytes(); layout and rounding stand in
    rra_serve.h)."""

    _size = staticmethod(kv8_page_bytes)
    _plan = "rra_kv8_attention_plan"

    def append(self, k, v, slots, stream=None) -> None:
        """Write k and v [tokens, kv_heads, head_dim] to the slots (int64; negative:
        skipped).  The slots of one block of 16 are neighbours in the list; the one at
        a block's start begins it anew, the others keep what it holds, rounded again
        where they are larger than all before."""
        st = _native.kv8_append(self._cache, self._dev, k, v, slots, stream)
        if st:
            raise rra.RraError(st, "rra_kv8_append")

    def read(self, slots, k, v, stream=None) -> None:
        """k and v [tokens, kv_heads, head_dim] become the values that the slots hold."""
        st = _native.kv8_read(self._cache, self._dev, k, v, slots, stream)
        if st:
            raise rra.RraError(st, "rra_kv8_read")

    def attention(self, q, out, cu_q, kv_len, block_table, *, max_q: int, max_kv: int, scale=None, causal: bool = True,
                  window: int = 0, lse=None, stream=None) -> None:
        """As KvCache.attention, over this cache (rra_kv8_attention); scores are below 2^26."""
        st = _native.kv8_attention(self._cache, self._dev, self._workspace, q, out, cu_q, kv_len, block_table, max_q, max_kv,
                                   self._scale if scale is None else scale, causal, window, lse, stream, self._home)
        if st:
            raise rra.RraError(st, "rra_kv8_attention")
