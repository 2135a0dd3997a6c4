"""Python binding of the decode-step operators (include/rra_serve.h).

Page bookkeeping, head norms with position rotation, a key/value cache held in
4 bits, and the attention over it: what a tensor-parallel rank runs around its
AllReduces.  As in rra.py this is argument checking and marshalling only; every
call enqueues one kernel of librra.so on the current stream (or `stream`), and
there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import rra

_SLOTS = struct.Struct("11P2q4i")
_ROPE = struct.Struct("9P10qd6i")
_TOKENS = struct.Struct("Pq4i3P5q2i")
_ATTN = struct.Struct("Pq4i7P6qd8i")

_I32, _I64, _F32, _BF16 = torch.int32, torch.int64, torch.float32, torch.bfloat16
_DTYPES = {_F32: 0, _BF16: 1}

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
               "rra_kv_attention_plan": [vp, ctypes.POINTER(ctypes.c_char_p)]}
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, ctypes.c_int
        lib.rra_kv_page_bytes.argtypes, lib.rra_kv_page_bytes.restype = [ctypes.c_int] * 3, ctypes.c_size_t
        lib.rra_kv_attention_workspace_bytes.argtypes = [ctypes.c_int]
        lib.rra_kv_attention_workspace_bytes.restype = ctypes.c_size_t
        _fns = lib
    return _fns


def _stream(stream, device):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _flat(name, t, dtype, n, device):
    """Pointer of a contiguous tensor of at least n elements."""
    if t.dtype is not dtype or t.get_device() != device or t.numel() < n or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of at least %d elements on cuda:%d" % (name, dtype, n, device))
    return t.data_ptr()


def _rows(name, t, dtype, shape, device):
    """Pointer, token stride and head stride of a [tokens, heads, channels] tensor whose channels are adjacent."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape:
        raise ValueError("%s must be a %s tensor of shape %s on cuda:%d" % (name, dtype, tuple(shape), device))
    a, b, c = t.stride()
    if c != 1:
        raise ValueError("%s: a head's channels must be adjacent" % name)
    # strides of a dimension of one element are never used
    return t.data_ptr(), a if shape[0] > 1 else shape[1] * shape[2] * 16, b if shape[1] > 1 else shape[2]


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
    dev = _device(seq_len)
    n = seq_len.numel()
    if block_table.dim() != 2 or block_table.shape[0] != n or block_table.dtype is not _I32 \
            or block_table.get_device() != dev or (block_table.numel() and block_table.stride(1) != 1):
        raise ValueError("block_table must be an int32 tensor [requests, pages] with adjacent pages")
    tokens = slots.numel()
    width = block_table.shape[1]
    args = _SLOTS.pack(
        _flat("seq_len", seq_len, _I32, n, dev), _flat("new_len", new_len, _I32, n, dev), block_table.data_ptr(),
        _flat("free_pages", free_pages, _I32, 0, dev), _flat("free_count", free_count, _I32, 1, dev),
        _flat("kv_len", kv_len, _I32, n, dev), _flat("cu_new", cu_new, _I32, n + 1, dev),
        _flat("slots", slots, _I64, 0, dev), _flat("positions", positions, _I32, tokens, dev),
        _flat("free_left", free_left, _I32, 1, dev), _flat("pages_short", pages_short, _I32, 1, dev),
        block_table.stride(0) if n > 1 else width, tokens, n, width, page_tokens, free_pages.numel())
    st = _lib().rra_slot_map(args, _stream(stream, dev))
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
    dev, dt = _device(q), q.dtype
    if dt not in _DTYPES:
        raise TypeError("unsupported dtype %s (float32, bfloat16)" % dt)
    if q.dim() != 3 or k.dim() != 3 or q.shape[0] != k.shape[0] or q.shape[2] != k.shape[2]:
        raise ValueError("q and k must be [tokens, heads, channels] with the same tokens and channels")
    t, hq, d = q.shape
    qp, qt, qh = _rows("q", q, dt, q.shape, dev)
    kp, kt, kh = _rows("k", k, dt, k.shape, dev)
    qo, qot, qoh = _rows("q_out", q_out, dt, q.shape, dev)
    ko, kot, koh = _rows("k_out", k_out, dt, k.shape, dev)
    rot = most = cp = sp = pp = 0
    if cos is not None:
        if cos.dim() != 2 or cos.shape != sin.shape:
            raise ValueError("cos and sin must be [max_position, rot/2]")
        most, rot = cos.shape[0], 2 * cos.shape[1]
        cp, sp = _flat("cos", cos, _F32, 0, dev), _flat("sin", sin, _F32, 0, dev)
        pp = _flat("positions", positions, _I32, t, dev)
    args = _ROPE.pack(qp, kp, qo, ko, 0 if q_weight is None else _flat("q_weight", q_weight, dt, d, dev),
                      0 if k_weight is None else _flat("k_weight", k_weight, dt, d, dev), cp, sp, pp,
                      qt, qh, kt, kh, qot, qoh, kot, koh, t, most, eps, hq, k.shape[1], d, rot, bool(interleaved),
                      _DTYPES[dt])
    st = _lib().rra_qk_norm_rope(args, _stream(stream, dev))
    if st:
        raise rra.RraError(st, "rra_qk_norm_rope")


def kv_page_bytes(page_tokens: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of one page of the 4-bit cache."""
    n = _lib().rra_kv_page_bytes(page_tokens, kv_heads, head_dim)
    if n == 0:
        raise rra.RraError(rra.ERR_INVALID_ARG, "rra_kv_page_bytes")
    return n


class KvCache:
    """A paged key/value cache held in 4 bits, in memory of the caller.

    `pages` is a contiguous uint8 CUDA tensor of whole pages (kv_page_bytes()
    each; their layout stands in rra_serve.h); it needs no initialisation.  The
    object holds the attention's workspace, so its attention() calls are ordered
    on one stream; append() and read() are not bound to it."""

    def __init__(self, pages, page_tokens: int, kv_heads: int, head_dim: int):
        lib = _lib()
        size = kv_page_bytes(page_tokens, kv_heads, head_dim)
        self._dev = _device(pages)
        if pages.dtype is not torch.uint8 or not pages.is_contiguous() or pages.numel() % size:
            raise ValueError("pages must be a contiguous uint8 tensor of whole pages (%d bytes each)" % size)
        self.pages = pages
        self.page_tokens, self.kv_heads, self.head_dim = int(page_tokens), int(kv_heads), int(head_dim)
        self.num_pages = pages.numel() // size
        self._workspace = torch.empty(lib.rra_kv_attention_workspace_bytes(head_dim), dtype=torch.uint8,
                                      device=pages.device)
        self._workspace[:_WORKSPACE_HEAD].zero_()
        self._head = (pages.data_ptr(), self.num_pages, self.page_tokens, self.kv_heads, self.head_dim, 0)

    def _tokens(self, fn, what, k, v, slots, stream):
        dt = k.dtype
        if dt not in _DTYPES:
            raise TypeError("unsupported dtype %s (float32, bfloat16)" % dt)
        shape = (slots.numel(), self.kv_heads, self.head_dim)
        kp, kt, kh = _rows("k", k, dt, shape, self._dev)
        vp, vt, vh = _rows("v", v, dt, shape, self._dev)
        args = _TOKENS.pack(*self._head, kp, vp, _flat("slots", slots, _I64, 0, self._dev), kt, kh, vt, vh, shape[0],
                            _DTYPES[dt], 0)
        st = fn(args, _stream(stream, self._dev))
        if st:
            raise rra.RraError(st, what)

    def append(self, k, v, slots, stream=None) -> None:
        """Write k and v [tokens, kv_heads, head_dim] to the slots (int64;
        negative: skipped)."""
        self._tokens(_lib().rra_kv_append, "rra_kv_append", k, v, slots, stream)

    def read(self, slots, k, v, stream=None) -> None:
        """k and v [tokens, kv_heads, head_dim] become the values that the slots hold."""
        self._tokens(_lib().rra_kv_read, "rra_kv_read", k, v, slots, stream)

    def _attention_args(self, q, out, cu_q, kv_len, block_table, max_q, max_kv, scale, causal, window, lse):
        dev = self._dev
        if q.dim() != 3 or q.shape[2] != self.head_dim or q.shape[1] % self.kv_heads:
            raise ValueError("q must be [tokens, heads, %d], heads a multiple of %d" % (self.head_dim, self.kv_heads))
        qp, qt, qh = _rows("q", q, _BF16, q.shape, dev)
        op, ot, oh = _rows("out", out, _BF16, q.shape, dev)
        n = kv_len.numel()
        if block_table.dim() != 2 or block_table.shape[0] != n or block_table.dtype is not _I32 \
                or block_table.get_device() != dev or (block_table.numel() and block_table.stride(1) != 1):
            raise ValueError("block_table must be an int32 tensor [requests, pages] with adjacent pages")
        t, hq, d = q.shape
        width = block_table.shape[1]
        return _ATTN.pack(
            *self._head, qp, op, 0 if lse is None else _flat("lse", lse, _F32, t * hq, dev),
            _flat("cu_q", cu_q, _I32, n + 1, dev), _flat("kv_len", kv_len, _I32, n, dev), block_table.data_ptr(),
            self._workspace.data_ptr(), qt, qh, ot, oh, block_table.stride(0) if n > 1 else width, t,
            1.0 / math.sqrt(d) if scale is None else scale, n, width, hq, max_q, max_kv, bool(causal), window, 0)

    def attention(self, q, out, cu_q, kv_len, block_table, *, max_q: int, max_kv: int, scale=None, causal: bool = True,
                  window: int = 0, lse=None, stream=None) -> None:
        """out = attention of q [tokens, q_heads, head_dim] (bfloat16) over the
        cache (rra_kv_attention).  Request b has the queries cu_q[b]..cu_q[b+1]
        and the first kv_len[b] tokens of its row of block_table, its own
        included; max_q and max_kv are what to plan for.  scale defaults to
        1/sqrt(head_dim).  lse: float32 [tokens, q_heads], optional."""
        args = self._attention_args(q, out, cu_q, kv_len, block_table, max_q, max_kv, scale, causal, window, lse)
        st = _lib().rra_kv_attention(args, _stream(stream, self._dev))
        if st:
            raise rra.RraError(st, "rra_kv_attention")

    def plan_kernel(self, q, out, cu_q, kv_len, block_table, *, max_q: int, max_kv: int, scale=None,
                    causal: bool = True, window: int = 0, lse=None) -> str:
        """Name of the kernel that attention() launches for these arguments."""
        args = self._attention_args(q, out, cu_q, kv_len, block_table, max_q, max_kv, scale, causal, window, lse)
        name = ctypes.c_char_p()
        st = _lib().rra_kv_attention_plan(args, ctypes.byref(name))
        if st:
            raise rra.RraError(st, "rra_kv_attention_plan")
        return name.value.decode()

    def status(self) -> int:
        """Status word of the attention calls so far (0 is fine); synchronises."""
        return int(self._workspace[:4].cpu().view(torch.int32).item())
