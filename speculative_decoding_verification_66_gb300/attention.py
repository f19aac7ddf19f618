"""Python binding of the paged cache and its attention (include/sv_attention.h):
the same names, torch tensors in.

Argument marshalling only, as in api.py. A cache is described by the tensors it
lies in:

    k_pages, v_pages  [pages, page_size, kv_heads, head_dim], bfloat16, float16
                      or float8_e4m3fn; any strides but the last (a cache with
                      its heads outermost in a page is a transposed view)
    k_exps, v_exps    [pages, page_size, kv_heads] uint8, e4m3 only
    page_table        [B, max_pages] int32
    cached_lens       [B] int32: tokens in the cache before this call's
    chunk_starts      [B + 1] int32: where each sequence's new tokens begin in
                      the packed arrays

Lengths and pages are read on the device only, so every call can be captured
into a CUDA graph and replayed with new ones.
"""
from __future__ import annotations

import ctypes
import struct
import threading
from contextlib import ExitStack
from functools import lru_cache

import torch

from . import _lib
from .api import SV_BF16, _check

SV_F16, SV_E4M3 = 2, 3
SV_SEQ_BAD_PAGE, SV_SEQ_BAD_LENGTH, SV_SEQ_OVERLAP = 16, 32, 64

_CODES = {torch.bfloat16: SV_BF16, torch.float16: SV_F16, torch.float8_e4m3fn: SV_E4M3}
# struct sv_paged_cache
_CACHE = struct.Struct("@4P12qq4iP2q2Pq")
_NO_EXPS = (0, 0, 0)


# (The checks below run at every step of a decode loop: plain ifs, messages built only when raised.)


def _require(ok, what):
    if not ok:
        raise ValueError(what)


def _cache(k_pages, v_pages, page_table, cached_lens, chunk_starts, k_exps, v_exps):
    """(packed struct sv_paged_cache, element type code, device, B)."""
    dev, dt, shape = k_pages.device, k_pages.dtype, k_pages.shape
    if len(shape) != 4 or not k_pages.is_cuda:
        raise ValueError("k_pages must be a CUDA tensor [pages, page_size, kv_heads, head_dim]")
    code = _CODES.get(dt)
    if code is None:
        raise TypeError(f"pages must be bfloat16, float16 or float8_e4m3fn, got {dt}")
    if v_pages.shape != shape or v_pages.dtype != dt or v_pages.device != dev:
        raise ValueError("v_pages must have k_pages' shape, dtype and device")
    ks, vs = k_pages.stride(), v_pages.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("pages must be contiguous along head_dim")
    if code == SV_E4M3:
        for e in (k_exps, v_exps):
            if e is None or e.dtype != torch.uint8 or e.shape != shape[:3] or e.device != dev:
                raise ValueError("k_exps and v_exps must be uint8 [pages, page_size, kv_heads] "
                                 "beside e4m3 pages")
        kep, vep, kes, ves = k_exps.data_ptr(), v_exps.data_ptr(), k_exps.stride(), v_exps.stride()
    elif k_exps is not None or v_exps is not None:
        raise ValueError("only e4m3 pages have exponents")
    else:
        kep, vep, kes, ves = 0, 0, _NO_EXPS, _NO_EXPS
    i32 = torch.int32
    if cached_lens.dim() != 1 or cached_lens.dtype != i32 or not cached_lens.is_contiguous() \
            or cached_lens.device != dev:
        raise ValueError("cached_lens must be contiguous int32 [B]")
    B = cached_lens.shape[0]
    table = page_table.shape
    if len(table) != 2 or table[0] != B or page_table.dtype != i32 or page_table.device != dev:
        raise ValueError("page_table must be int32 [B, max_pages]")
    row, step = page_table.stride()
    if (step != 1 and table[1] > 1) or (B > 1 and row < table[1]):
        raise ValueError("page_table's rows must be contiguous and must not overlap")
    if chunk_starts.shape != (B + 1,) or chunk_starts.dtype != i32 \
            or not chunk_starts.is_contiguous() or chunk_starts.device != dev:
        raise ValueError("chunk_starts must be contiguous int32 [B + 1]")
    packed = _CACHE.pack(
        k_pages.data_ptr(), v_pages.data_ptr(), kep, vep, ks[0], vs[0], ks[1], vs[1], ks[2], vs[2],
        kes[0], ves[0], kes[1], ves[1], kes[2], ves[2], shape[0], shape[1], shape[2], shape[3],
        code, page_table.data_ptr(), max(row, table[1]), table[1], cached_lens.data_ptr(),
        chunk_starts.data_ptr(), B)
    return packed, code, dev, B


def _rows(x, name, heads, head_dim, dev, cache_code):
    """Type code of a packed array [tokens, heads, head_dim]."""
    code = _CODES.get(x.dtype)
    if code is None or code == SV_E4M3 or (cache_code != SV_E4M3 and code != cache_code):
        raise TypeError(f"{name} must be bfloat16 or float16, and of the cache's type unless that "
                        f"is e4m3, got {x.dtype}")
    shape = x.shape
    if len(shape) != 3 or shape[2] != head_dim or (heads is not None and shape[1] != heads) \
            or x.device != dev:
        raise ValueError(f"{name} must be [tokens, heads, head_dim] on the cache's device")
    if x.stride(2) != 1 and x.numel() > 0:
        raise ValueError(f"{name} must be contiguous along head_dim")
    return code


def _status(seq_status, B, dev):
    if seq_status is None:
        return None
    _require(seq_status.dtype == torch.int32 and seq_status.shape == (B,)
             and seq_status.is_contiguous() and seq_status.device == dev,
             "seq_status must be contiguous int32 [B]")
    return seq_status.data_ptr()


def _on(dev, stream, call, tensors):
    """call(raw stream) with dev and stream current, so that what it allocates belongs to the
    stream the kernels run on. The allocator is told of tensors used on a stream not their own."""
    if torch.cuda.current_device() == dev.index and stream is None:
        # (the handle of the current stream, without building a Stream object)
        return call(torch._C._cuda_getCurrentRawStream(dev.index))
    with ExitStack() as stack:
        if torch.cuda.current_device() != dev.index:
            stack.enter_context(torch.cuda.device(dev))
        if stream is not None and stream != torch.cuda.current_stream(dev):
            stack.enter_context(torch.cuda.stream(stream))
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
        return call(torch._C._cuda_getCurrentRawStream(dev.index))


_kept = threading.local()


def _workspace(dev, stream, nbytes):
    """At least nbytes, kept for this thread's calls on this stream, which the stream puts in
    order. A call that is being captured gets a buffer of its own, from the graph's pool: its
    replays may run beside anything."""
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    kept = _kept.__dict__
    w = kept.get((dev.index, stream))
    if w is None or w.numel() < nbytes:
        w = kept[(dev.index, stream)] = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return w


def sv_kv_append(key, value, k_pages, v_pages, page_table, cached_lens, chunk_starts, *,
                 k_exps=None, v_exps=None, seq_status=None, stream=None) -> None:
    """Write the new tokens' key and value [tokens, kv_heads, head_dim] (any strides but the last)
    into the cache, quantised where it is e4m3. Asynchronous on ``stream`` (default: the current
    stream of the pages' device)."""
    cache, code, dev, B = _cache(k_pages, v_pages, page_table, cached_lens, chunk_starts, k_exps,
                                 v_exps)
    _, _, H, D = k_pages.shape
    dtype = _rows(key, "key", H, D, dev, code)
    _rows(value, "value", H, D, dev, code)
    if value.shape != key.shape or value.dtype != key.dtype:
        raise ValueError("value must have key's shape and dtype")
    status = _status(seq_status, B, dev)
    ks, vs = key.stride(), value.stride()

    def call(s):
        _check(_lib.load_attention().sv_kv_append(
            cache, key.data_ptr(), value.data_ptr(), dtype, key.shape[0], ks[0], ks[1], vs[0],
            vs[1], status, s), "sv_kv_append")

    _on(dev, stream, call, (key, value, k_pages, v_pages, page_table, cached_lens, chunk_starts,
                            k_exps, v_exps, seq_status))


def sv_kv_read(k_pages, v_pages, page_table, cached_lens, chunk_starts, tokens: int, *,
               k_exps=None, v_exps=None, dtype=None, key=None, value=None, seq_status=None,
               stream=None):
    """Read positions cached_lens[b] .. cached_lens[b] + (chunk_starts[b + 1] - chunk_starts[b])
    of every sequence back. Returns (key, value) [tokens, kv_heads, head_dim] of ``dtype``
    (default: the cache's, bfloat16 from e4m3); ``tokens`` is chunk_starts[B], which the host has
    to know."""
    cache, code, dev, B = _cache(k_pages, v_pages, page_table, cached_lens, chunk_starts, k_exps,
                                 v_exps)
    _, _, H, D = k_pages.shape
    if dtype is None:
        dtype = key.dtype if key is not None else \
            torch.bfloat16 if code == SV_E4M3 else k_pages.dtype
    status = _status(seq_status, B, dev)
    _require(tokens >= 0, "tokens must not be negative")

    def call(s):
        out = []
        for name, x in (("key", key), ("value", value)):
            if x is None:
                x = torch.empty((tokens, H, D), dtype=dtype, device=dev)
            elif x.shape[0] != tokens or x.dtype != dtype or not x.is_contiguous():
                raise ValueError(f"{name} must be contiguous [tokens, kv_heads, head_dim] of dtype")
            out.append(x)
            d = _rows(x, name, H, D, dev, code)
        _check(_lib.load_attention().sv_kv_read(cache, out[0].data_ptr(), out[1].data_ptr(), d,
                                                tokens, status, s), "sv_kv_read")
        return tuple(out)

    return _on(dev, stream, call, (key, value, k_pages, v_pages, page_table, cached_lens,
                                   chunk_starts, k_exps, v_exps, seq_status))


@lru_cache(maxsize=256)
def sv_chunk_attention_workspace_bytes(B: int, tokens: int, q_heads: int, kv_heads: int,
                                       head_dim: int, max_chunk: int = 0) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.load_attention().sv_chunk_attention_workspace_bytes(
        B, tokens, q_heads, kv_heads, head_dim, max_chunk, ctypes.byref(n)),
        "sv_chunk_attention_workspace_bytes")
    return n.value


def sv_chunk_attention(query, k_pages, v_pages, page_table, cached_lens, chunk_starts, *,
                       k_exps=None, v_exps=None, scale=None, window: int = 0, max_chunk: int = 0,
                       out=None, lse=None, return_lse: bool = False, seq_status=None,
                       workspace=None, stream=None):
    """Attention of the new tokens' query [tokens, q_heads, head_dim] over their sequences' caches,
    which hold the new tokens too (``sv_kv_append`` first): query t of sequence b sees positions up
    to its own, cached_lens[b] + t, and with a ``window`` only the last ``window`` of them.

    ``scale`` defaults to head_dim ** -0.5. ``max_chunk``: an upper bound of the sequences' new
    tokens (0: tokens); a tight one lets the launches be planned for it (512 single tokens take half
    as long again without). A workspace (up to 43 MB) is kept for the thread and stream
    unless one is given (``sv_chunk_attention_workspace_bytes``). Returns out, or (out, lse)
    with ``return_lse`` or an ``lse`` tensor (float32 [tokens, q_heads])."""
    return _attention(query, k_pages, v_pages, page_table, cached_lens, chunk_starts, k_exps, v_exps,
                      scale, window, max_chunk, out, lse, return_lse, seq_status, workspace, stream)


def sv_chunk_attention_gated(query, k_pages, v_pages, page_table, cached_lens, chunk_starts, gate, *,
                             block: int = -1, k_exps=None, v_exps=None, scale=None,
                             window: int = 0, max_chunk: int = 0, stream=None) -> dict:
    """Test hook for the timeout path: sv_chunk_attention with the values' loads of one thread
    ``block`` (negative: all) held until the device int32 ``gate`` (one element) is nonzero.
    Returns out, lse and seq_status."""
    if gate.dtype != torch.int32 or not gate.is_cuda or gate.numel() < 1:
        raise ValueError("gate must be an int32 CUDA tensor")
    status = torch.empty(cached_lens.shape, dtype=torch.int32, device=query.device)
    out, lse = _attention(query, k_pages, v_pages, page_table, cached_lens, chunk_starts, k_exps,
                          v_exps, scale, window, max_chunk, None, None, True, status, None, stream,
                          (int(block), gate))
    return {"out": out, "lse": lse, "seq_status": status}


def _attention(query, k_pages, v_pages, page_table, cached_lens, chunk_starts, k_exps, v_exps, scale,
               window, max_chunk, out, lse, return_lse, seq_status, workspace, stream, gate=None):
    cache, code, dev, B = _cache(k_pages, v_pages, page_table, cached_lens, chunk_starts, k_exps,
                                 v_exps)
    _, _, H, D = k_pages.shape
    dtype = _rows(query, "query", None, D, dev, code)
    N, Hq, _ = query.shape
    if H < 1 or Hq < 1 or Hq % H != 0:
        raise ValueError("query heads must be a multiple of kv_heads")
    status = _status(seq_status, B, dev)
    if scale is None:
        scale = D ** -0.5
    if out is not None:
        _require(out.shape == query.shape and out.dtype == query.dtype and out.device == dev and
                 out.is_contiguous(), "out must be contiguous, of query's shape, dtype and device")
    if lse is not None:
        _require(lse.shape == (N, Hq) and lse.dtype == torch.float32 and lse.device == dev
                 and lse.is_contiguous(), "lse must be contiguous float32 [tokens, q_heads]")
    if workspace is not None:
        _require(workspace.device == dev and workspace.dtype == torch.uint8 and
                 workspace.is_contiguous(), "workspace must be contiguous uint8 on the device")
    qs = query.stride()

    def call(s):
        o = out
        if o is None:
            o = torch.empty_like(query) if query.is_contiguous() else \
                torch.empty((N, Hq, D), dtype=query.dtype, device=dev)
        z = torch.empty((N, Hq), dtype=torch.float32, device=dev) if lse is None and return_lse \
            else lse
        w = workspace
        if w is None:
            w = _workspace(dev, s, sv_chunk_attention_workspace_bytes(B, N, Hq, H, D, max_chunk))
        args = (cache, query.data_ptr(), dtype, N, Hq, qs[0], qs[1], scale, window, max_chunk,
                o.data_ptr(), None if z is None else z.data_ptr(), status, w.data_ptr(), w.numel(),
                s)
        if gate is None:
            _check(_lib.load_attention().sv_chunk_attention(*args), "sv_chunk_attention")
        else:
            _check(_lib.load_attention().sv_chunk_attention_gated(
                *args, gate[0], gate[1].data_ptr()), "sv_chunk_attention_gated")
        return o if z is None else (o, z)

    return _on(dev, stream, call, (query, k_pages, v_pages, page_table, cached_lens, chunk_starts,
                                   k_exps, v_exps, out, lse, seq_status, workspace,
                                   None if gate is None else gate[1]))
