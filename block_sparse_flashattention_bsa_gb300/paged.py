"""Serving over a paged key/value cache: write new tokens, attend with one or
a tree of drafted tokens per sequence, keep the accepted ones, and the pages.

Pools are bf16 [n_pages, Hkv, page, D] (one layer) or [layers, n_pages, Hkv,
page, D]; a page is a key block of the attention, page in {64, 128}.
page_table is int32 [n_seqs, max_pages] with -1 behind a sequence's pages,
page_ref int32 [n_pages] counts the table entries that hold a page (0: free).

Marshalling only; contracts are in ``include/bsa.h``, the kernels in
``csrc/bsa_rope.cu`` (append), ``csrc/bsa_tree.cu`` and ``csrc/bsa_cache.cu``.
"""

from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from ._binding import _PageCache, _TreeArgs, _addr, _check, _same_device, _scope, _stream, lib
from .rope import _outputs, _side_args


def _pool(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor, layers: bool) -> _PageCache:
    if k_cache.shape != v_cache.shape or k_cache.dim() not in ((4, 5) if layers else (4,)):
        raise ValueError("expected k_cache and v_cache of one shape [n_pages, Hkv, page, D]%s"
                         % (" or [layers, n_pages, Hkv, page, D]" if layers else ""))
    for t in (k_cache, v_cache):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError("expected contiguous bf16 caches")
    _ints("page_table", page_table, None)
    if page_table.dim() != 2:
        raise ValueError("page_table: int32 [n_seqs, max_pages]")
    n_pages, Hkv, page, D = k_cache.shape[-4:]
    return _PageCache(_addr(k_cache), _addr(v_cache), k_cache.shape[0] if k_cache.dim() == 5 else 1, n_pages, Hkv,
                      page, D, _addr(page_table), page_table.shape[0], page_table.shape[1])


def _ints(name: str, t: torch.Tensor, shape, dtype=torch.int32) -> None:
    if t.dtype != dtype or not t.is_contiguous() or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError("%s: contiguous %s%s" % (name, dtype, "" if shape is None else " %s" % (tuple(shape),)))


def cache_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 page_table: torch.Tensor, seq_ids: torch.Tensor, slots: torch.Tensor,
                 inv_freq: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 gain: float = 1.0, interleaved: bool = False, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """`qk_norm_rope` for new tokens of a served batch: token i (q [tokens,Hq,D],
    k, v [tokens,Hkv,D], any strides) belongs to slot slots[i] of sequence
    seq_ids[i] (< 0: padding, skipped), and its rotated key and its value go to
    that slot's page.  positions default to the slots (a tree's drafts give
    their depth).  Returns the rotated queries [tokens,Hq,D]."""
    a, device, _, N, Hq, Hkv, D = _side_args(q, k, v, inv_freq, positions, q_weight, k_weight, eps, gain,
                                             interleaved, 1, 1)
    c = _pool(k_cache, v_cache, page_table, False)
    _same_device(q, k_cache, v_cache, page_table, seq_ids, slots)
    if v is None or k_cache.shape[1] != Hkv or k_cache.shape[3] != D:
        raise ValueError("k and v need the cache's heads and head size")
    _ints("seq_ids", seq_ids, (N,))
    _ints("slots", slots, (N,))
    with _scope(device, stream):
        oq, = _outputs(None if out is None else (out,), [(N, Hq, D)], q)
        _check("bsa_cache_append", lib().bsa_cache_append(ctypes.byref(a), ctypes.byref(c), _addr(seq_ids),
                                                          _addr(slots), _addr(oq), _stream(None)))
    return oq


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                   context_len: torch.Tensor, draft_len: Optional[torch.Tensor] = None,
                   tree_mask: Optional[torch.Tensor] = None, row_ptr: Optional[torch.Tensor] = None,
                   col_idx: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                   out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of the T drafted tokens of each sequence (T = 1: decoding) over
    its pages: q [B,T,Hq,D] bf16, draft t in slot context_len[b] + t, attending
    to the committed slots and to the drafts in the bits of tree_mask[b][t]
    (int64 [B,T]; None: a chain).  draft_len int32 [B] (None: T): rows behind
    it are left as they were.  row_ptr [B*Hkv+1], col_idx: only the listed
    logical pages of each (sequence, key head).

    Returns (O bf16 [B,T,Hq,D], LSE fp32 [B,T,Hq])."""
    if q.dim() != 4 or q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q: contiguous bf16 [B, T, Hq, D]")
    B, T, Hq, D = q.shape
    c = _pool(k_cache, v_cache, page_table, False)
    device = _same_device(q, k_cache, v_cache, page_table, context_len, draft_len, tree_mask, row_ptr, col_idx, out,
                          lse)
    if page_table.shape[0] != B or k_cache.shape[3] != D:
        raise ValueError("page_table needs one row per sequence, the caches q's head size")
    _ints("context_len", context_len, (B,))
    if draft_len is not None:
        _ints("draft_len", draft_len, (B,))
    if tree_mask is not None:
        _ints("tree_mask", tree_mask, (B, T), torch.int64)
    if (row_ptr is None) != (col_idx is None):
        raise ValueError("row_ptr and col_idx come together")
    if row_ptr is not None:
        _ints("row_ptr", row_ptr, (B * c.Hkv + 1,))
        _ints("col_idx", col_idx, None)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with _scope(device, stream):
        o, = _outputs(None if out is None else (out,), [(B, T, Hq, D)], q)
        if lse is None:
            lse = torch.empty((B, T, Hq), dtype=torch.float32, device=device)
        _ints("lse", lse, (B, T, Hq), torch.float32)
        n = int(lib().bsa_tree_attention_workspace(B, T, Hq, c.Hkv, D))
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        # an empty list has no storage: any address does, nothing below its capacity of 0 is read
        ci = None if col_idx is None else (col_idx.data_ptr() or row_ptr.data_ptr())
        a = _TreeArgs(B, T, Hq, _addr(q), _addr(context_len), _addr(draft_len), _addr(tree_mask), _addr(row_ptr),
                      ci, 0 if col_idx is None else col_idx.numel(), _addr(o), _addr(lse), float(scale))
        _check("bsa_tree_attention", lib().bsa_tree_attention(ctypes.byref(a), ctypes.byref(c), _addr(ws), n,
                                                              _stream(None)))
    return o, lse


def cache_accept(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor, context_len: torch.Tensor,
                 accepted: torch.Tensor, n_accepted: torch.Tensor, new_len: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """Moves the rows of the accepted drafts (accepted int32 [n_seqs,T], the
    first n_accepted[b] strictly increasing) up behind the committed slots, in
    every layer of the pools; returns the new lengths context_len + n_accepted."""
    c = _pool(k_cache, v_cache, page_table, True)
    device = _same_device(k_cache, v_cache, page_table, context_len, accepted, n_accepted, new_len)
    S = page_table.shape[0]
    if accepted.dim() != 2:
        raise ValueError("accepted: int32 [n_seqs, T]")
    _ints("context_len", context_len, (S,))
    _ints("accepted", accepted, (S, accepted.shape[1]))
    _ints("n_accepted", n_accepted, (S,))
    with _scope(device, stream):
        if new_len is None:
            new_len = torch.empty_like(context_len)
        _ints("new_len", new_len, (S,))
        _check("bsa_cache_accept", lib().bsa_cache_accept(
            ctypes.byref(c), _addr(context_len), _addr(accepted), _addr(n_accepted), accepted.shape[1],
            _addr(new_len), _stream(None)))
    return new_len


def _request(fn: str, page_table, page_ref, a, b, n, k_cache, v_cache, stream) -> torch.Tensor:
    c = _pool(k_cache, v_cache, page_table, True)
    device = _same_device(k_cache, v_cache, page_table, page_ref, a, b, n)
    _ints("page_ref", page_ref, (c.n_pages,))
    if a.dim() != 1:
        raise ValueError("requests: int32 vectors of one length")
    for t in (a, b, n):
        _ints("requests", t, a.shape)
    N = a.numel()
    with _scope(device, stream):
        granted = torch.empty(N, dtype=torch.int32, device=device)
        if N == 0:
            return granted
        size = int(lib().bsa_cache_pages_workspace(N, c.n_seqs, c.n_pages))
        ws = torch.empty(size, dtype=torch.uint8, device=device)
        _check("bsa_" + fn, getattr(lib(), "bsa_" + fn)(
            ctypes.byref(c), _addr(page_ref), N, _addr(a), _addr(b), _addr(n), _addr(granted), _addr(ws), size,
            _stream(None)))
    return granted


def cache_resize(page_table: torch.Tensor, page_ref: torch.Tensor, seqs: torch.Tensor, keep: torch.Tensor,
                 capacity: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, stream=None) -> torch.Tensor:
    """Sequence seqs[i] keeps its first keep[i] slots and holds pages for
    capacity[i] of them (0, 0 frees it); from slot keep[i] on its pages are its
    own.  Updates page_table and page_ref (and copies the kept rows of a shared
    part-filled page); returns int32 1 (served) or 0 (refused) per request."""
    return _request("cache_resize", page_table, page_ref, seqs, keep, capacity, k_cache, v_cache, stream)


def cache_fork(page_table: torch.Tensor, page_ref: torch.Tensor, src: torch.Tensor, dst: torch.Tensor,
               lens: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, stream=None) -> torch.Tensor:
    """Sequence dst[i] (which holds no page) gets the first lens[i] slots of
    src[i]: full pages shared, the rows of a part-filled last page copied.
    Returns int32 1 (served) or 0 (refused) per request."""
    return _request("cache_fork", page_table, page_ref, src, dst, lens, k_cache, v_cache, stream)


def cache_compact(page_table: torch.Tensor, page_ref: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  stream=None) -> torch.Tensor:
    """Moves the live pages to the front of the pool, table and counts with
    them; returns int32 [n_pages]: where each page went, -1 for free ones."""
    c = _pool(k_cache, v_cache, page_table, True)
    device = _same_device(k_cache, v_cache, page_table, page_ref)
    _ints("page_ref", page_ref, (c.n_pages,))
    with _scope(device, stream):
        new_page = torch.empty_like(page_ref)
        size = int(lib().bsa_cache_pages_workspace(0, c.n_seqs, c.n_pages))
        ws = torch.empty(size, dtype=torch.uint8, device=device)
        _check("bsa_cache_compact", lib().bsa_cache_compact(ctypes.byref(c), _addr(page_ref), _addr(new_page),
                                                            _addr(ws), size, _stream(None)))
    return new_page
