"""Answering with a model: the paged cache of keys and values (include/s2attn.h).

A step appends its new tokens' keys and values and attends from the new tokens
over everything their sequences hold:

    cache = KVCache.empty(pages, page_size, heads, dim)          # bits=4 packs rows to 4 bits
    batch = CacheBatch(page_table, seq_lens, q_starts, tokens)   # device int32 tensors
    q = cache_append(cache, batch, k, v, q)                      # rotates q and k on the way
    o = cache_attention(cache, batch, q)

Argument marshalling only; the computation runs in libs2attn.so.  Tensors that
a call allocates itself belong to the stream that it runs on.  There is no
backward: tensors that want a gradient are refused outside torch.no_grad().
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import binding
from .binding import _check, _ptr, lib

# The current stream's handle without the object around it, and the current device: a step's calls are short enough
# for the host's time to count (the helpers below look at each tensor once and pass plain numbers on).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

CACHE_BF16, CACHE_Q4 = 0, 1


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("D", ctypes.c_int64), ("format", ctypes.c_int)]


class _BatchStruct(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p), ("q_starts", ctypes.c_void_p),
                ("seqs", ctypes.c_int64), ("tokens", ctypes.c_int64), ("table_width", ctypes.c_int64),
                ("max_new", ctypes.c_int64), ("max_len", ctypes.c_int64)]


class KVCache:
    """Pages of keys and values: k, v bf16 [pages, heads, page_size, D], or for a 4-bit cache uint8
    [pages, heads, page_size, D/2] with k_scale, v_scale bf16 [pages, heads, page_size, 2]."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        q4 = k_scale is not None
        tensors = [k, v] + ([k_scale, v_scale] if q4 else [])
        if (v_scale is not None) != q4:
            raise ValueError("k_scale and v_scale go together")
        for t in tensors:
            if t.dim() != 4 or not t.is_cuda or not t.is_contiguous() or t.device != k.device:
                raise ValueError("expected contiguous CUDA tensors [pages, heads, page_size, ..] on one device")
        if any(t.dtype != (torch.uint8 if q4 else torch.bfloat16) for t in (k, v)) or v.shape != k.shape:
            raise ValueError("k and v must be of one shape, bf16 (or uint8 codes with scales)")
        if q4 and any(t.dtype != torch.bfloat16 or t.shape != (*k.shape[:3], 2) for t in (k_scale, v_scale)):
            raise ValueError("k_scale and v_scale must be bf16 [pages, heads, page_size, 2]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.heads, self.page_size = (int(x) for x in k.shape[:3])
        self.dim = int(k.shape[3]) * (2 if q4 else 1)
        self.format = CACHE_Q4 if q4 else CACHE_BF16
        self.device, self.index = k.device, k.device.index
        self._struct = _CacheStruct(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), self.pages, self.heads,
                                    self.page_size, self.dim, self.format)
        self.address = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, pages: int, page_size: int, heads: int, dim: int, bits: int = 16, device="cuda"):
        if bits not in (4, 16):
            raise ValueError("bits must be 16 or 4")
        shape, kind = (pages, heads, page_size, dim), torch.bfloat16
        if bits == 4:
            shape, kind = (pages, heads, page_size, dim // 2), torch.uint8
        data = [torch.empty(shape, dtype=kind, device=device) for _ in range(2)]
        scales = [torch.empty((*shape[:3], 2), dtype=torch.bfloat16, device=device) for _ in range(2 if bits == 4 else 0)]
        return cls(*data, *scales)


class CacheBatch:
    """The sequences of a call: page_table int32 [seqs, width], seq_lens int32 [seqs] (new tokens included) and
    q_starts int32 [seqs + 1], the packed starts of the new tokens (None: one per sequence), on the device;
    tokens: length of the packed axis.  max_new, max_len: the host's bounds of a sequence's new tokens and length, if
    known; they choose kernels, and change results by no more than the rounding of weights to bf16.  The tensors'
    contents are read when kernels run: the same batch serves step after step, and captured graphs, while the program
    updates them in place."""

    def __init__(self, page_table, seq_lens, q_starts=None, tokens: int | None = None, max_new: int = 0,
                 max_len: int = 0):
        for t, dims in ((page_table, 2), (seq_lens, 1), (q_starts, 1)):
            if t is not None and (t.dim() != dims or t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous()
                                  or t.device != page_table.device):
                raise ValueError("page_table [seqs, width], seq_lens [seqs] and q_starts [seqs + 1] must be contiguous "
                                 "CUDA int32 tensors on one device")
        seqs, width = (int(x) for x in page_table.shape)
        if seq_lens.shape != (seqs,) or (q_starts is not None and q_starts.shape != (seqs + 1,)):
            raise ValueError("page_table [seqs, width], seq_lens [seqs] and q_starts [seqs + 1] do not fit")
        if tokens is None:
            if q_starts is not None:
                raise ValueError("with q_starts, tokens (the length of the packed axis) must be given")
            tokens = seqs
        self.page_table, self.seq_lens, self.q_starts = page_table, seq_lens, q_starts
        self.seqs, self.tokens, self.index = seqs, int(tokens), page_table.device.index
        self._struct = _BatchStruct(_ptr(page_table), _ptr(seq_lens), _ptr(q_starts), seqs, self.tokens, width,
                                    int(max_new), int(max_len))
        self.address = ctypes.addressof(self._struct)


def _stream(stream, cache) -> int:
    return _raw_stream(cache.index) if stream is None else binding._stream(stream)


# ------------------------------------------------------------------ raw entry points (same names as the C ABI)


def s2attn_cache_append(cache, batch, q, ldq, k, ldk, v, ldv, q_out, heads, positions, base, scale, stream=None) -> int:
    return lib().s2attn_cache_append(cache.address, batch.address, _ptr(q), ldq, _ptr(k), ldk, _ptr(v), ldv,
                                     _ptr(q_out), heads, _ptr(positions), base, scale, _stream(stream, cache))


def s2attn_cache_read(cache, batch, k_out, v_out, stream=None) -> int:
    return lib().s2attn_cache_read(cache.address, batch.address, _ptr(k_out), _ptr(v_out), _stream(stream, cache))


def s2attn_cache_attn_workspace_size(cache, batch, heads) -> int:
    return int(lib().s2attn_cache_attn_workspace_size(cache.address, batch.address, heads))


def s2attn_cache_attn(cache, batch, q, ldq, o, lse, heads, workspace, workspace_bytes, stream=None) -> int:
    return lib().s2attn_cache_attn(cache.address, batch.address, _ptr(q), ldq, _ptr(o), _ptr(lse), heads,
                                   _ptr(workspace), workspace_bytes, _stream(stream, cache))


# ------------------------------------------------------------------ tensor-level helpers


@contextlib.contextmanager
def _on(device, stream):
    """The cache's device and the call's stream as the current ones, so that what is allocated inside belongs to it."""
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device)
            with torch.cuda.stream(s):
                yield


def _plain(cache, batch, stream):
    """Whether there is nothing to switch: the call runs on the current stream of the cache's device."""
    if batch.index != cache.index:
        raise ValueError("the batch is on another device than the cache")
    return stream is None and cache.index == _current_device()


def _rows(name, t, cache, batch, heads):
    """Row stride of [tokens, heads, D] bf16 rows whose heads lie side by side."""
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError("%s wants a gradient, and there is none through the cache: call under torch.no_grad()" % name)
    if t.dtype is not torch.bfloat16 or t.get_device() != cache.index or t.shape != (batch.tokens, heads, cache.dim):
        raise ValueError("%s must be bf16 [%d, %d, %d] on the cache's device" % (
            name, batch.tokens, heads, cache.dim))
    row, head, one = t.stride()
    if one != 1 or (head != cache.dim and heads > 1):
        raise ValueError("the heads of a token of %s must lie side by side" % name)
    return row if batch.tokens > 1 else heads * cache.dim  # (of one token any stride will do)


def _query_heads(q):
    if q.dim() != 3:
        raise ValueError("q must be bf16 [tokens, heads, D]")
    return q.shape[1]


def _whole(name, t, shape, cache, dtype=torch.bfloat16):
    if t.dtype is not dtype or t.shape != shape or t.get_device() != cache.index or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor %s on the cache's device" % (name, dtype, tuple(shape)))


def cache_append(cache: KVCache, batch: CacheBatch, k, v, q=None, positions=None, base: float = 10000.0,
                 scale: float = 1.0, out=None, stream=None):
    """Stores the new tokens' keys (rotated to their positions) and values [tokens, cache.heads, D]; returns the
    rotated queries if q [tokens, heads, D] is given.  base=0: the keys are stored as they are."""
    if not _plain(cache, batch, stream):
        with _on(cache.device, stream):
            return cache_append(cache, batch, k, v, q, positions, base, scale, out)
    ldk, ldv = _rows("k", k, cache, batch, cache.heads), _rows("v", v, cache, batch, cache.heads)
    ldq = heads = 0
    if q is not None:
        heads = _query_heads(q)
        ldq = _rows("q", q, cache, batch, heads)
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        else:
            _whole("out", out, q.shape, cache)
    elif out is not None:
        raise ValueError("out goes with q")
    if positions is not None:
        _whole("positions", positions, (batch.tokens,), cache, torch.int32)
    _check(lib().s2attn_cache_append(
        cache.address, batch.address, None if q is None else q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv,
        None if q is None else out.data_ptr(), heads, None if positions is None else positions.data_ptr(), base, scale,
        _raw_stream(cache.index)))
    return out


def cache_read(cache: KVCache, batch: CacheBatch, out=None, stream=None):
    """The rows of the batch's new tokens back as bf16 (k, v) [tokens, cache.heads, D]; tokens without a row are left
    as they were in ``out``, an optional preallocated pair."""
    if not _plain(cache, batch, stream):
        with _on(cache.device, stream):
            return cache_read(cache, batch, out)
    shape = (batch.tokens, cache.heads, cache.dim)
    if out is None:
        k, v = (torch.empty(shape, dtype=torch.bfloat16, device=cache.device) for _ in range(2))
    else:
        k, v = out
        _whole("out", k, shape, cache)
        _whole("out", v, shape, cache)
    _check(lib().s2attn_cache_read(cache.address, batch.address, k.data_ptr(), v.data_ptr(), _raw_stream(cache.index)))
    return k, v


def cache_attention_workspace(cache: KVCache, batch: CacheBatch, heads: int):
    """A workspace for cache_attention, to keep over steps: it serves every batch and number of heads over caches of this
    many channels.  Calls that may overlap on the GPU need one each."""
    n = s2attn_cache_attn_workspace_size(cache, batch, heads)
    if n == 0:
        raise ValueError("%d heads, this cache and this batch do not go together: %s" % (
            heads, binding.s2attn_last_error()))
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def cache_attention(cache: KVCache, batch: CacheBatch, q, out=None, lse=None, workspace=None, stream=None):
    """Attention of the new tokens' queries [tokens, heads, D] (rotated) over their sequences up to themselves; returns
    o [tokens, heads, D].  lse: optional float32 [tokens, heads] to fill.  Without a workspace one is allocated."""
    if not _plain(cache, batch, stream):
        with _on(cache.device, stream):
            return cache_attention(cache, batch, q, out, lse, workspace)
    heads = _query_heads(q)
    ldq = _rows("q", q, cache, batch, heads)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    else:
        _whole("out", out, q.shape, cache)
    if lse is not None:
        _whole("lse", lse, q.shape[:2], cache, torch.float32)
    if workspace is None:
        workspace = cache_attention_workspace(cache, batch, heads)
    elif workspace.get_device() != cache.index or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous on the cache's device")
    _check(lib().s2attn_cache_attn(
        cache.address, batch.address, q.data_ptr(), ldq, out.data_ptr(), None if lse is None else lse.data_ptr(), heads,
        workspace.data_ptr(), workspace.nbytes, _raw_stream(cache.index)))
    return out
