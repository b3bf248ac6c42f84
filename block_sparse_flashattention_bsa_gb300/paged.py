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

import math
import struct
from typing import Optional, Tuple

import torch

from ._binding import _addr, _check, _raw_stream, _same_device, _scope, lib
from .rope import _output, _side_args

_BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
_CACHE = struct.Struct("@2P5iP2i")    # bsa_page_cache
_TREE = struct.Struct("@3i6Pq2Pf")    # bsa_tree_args


def _pool(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor, layers: bool):
    """Packed bsa_page_cache and the pool's (n_pages, Hkv, page, D, n_seqs)."""
    ks, ts = k_cache.shape, page_table.shape
    if ks != v_cache.shape or len(ks) not in ((4, 5) if layers else (4,)):
        raise ValueError("expected k_cache and v_cache of one shape [n_pages, Hkv, page, D]%s"
                         % (" or [layers, n_pages, Hkv, page, D]" if layers else ""))
    if k_cache.dtype is not _BF16 or v_cache.dtype is not _BF16 or not k_cache.is_contiguous() \
            or not v_cache.is_contiguous():
        raise ValueError("expected contiguous bf16 caches")
    if page_table.dtype is not _I32 or len(ts) != 2 or not page_table.is_contiguous():
        raise ValueError("page_table: contiguous int32 [n_seqs, max_pages]")
    n_pages, Hkv, page, D = ks[-4:]
    return (_CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), ks[0] if len(ks) == 5 else 1, n_pages, Hkv, page, D,
                        page_table.data_ptr(), ts[0], ts[1]), n_pages, Hkv, page, D, ts[0])


def _ints(name: str, t: torch.Tensor, shape, dtype=_I32) -> None:
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s: contiguous %s %s" % (name, dtype, shape))


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
    a, index, _, N, Hq, Hkv, D = _side_args(q, k, v, inv_freq, positions, q_weight, k_weight, eps, gain,
                                            interleaved, 1, False)
    c, _, heads, _, width, _ = _pool(k_cache, v_cache, page_table, False)
    _same_device(q, k_cache, v_cache, page_table, seq_ids, slots)
    if v is None or heads != Hkv or width != D:
        raise ValueError("k and v need the cache's heads and head size")
    _ints("seq_ids", seq_ids, (N,))
    _ints("slots", slots, (N,))
    with _scope(index, stream):
        out = _output(out, (N, Hq, D), q)
        st = lib().bsa_cache_append(a, c, seq_ids.data_ptr(), slots.data_ptr(), out.data_ptr(), _raw_stream(index))
    if st:
        _check("bsa_cache_append", st)
    return out


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
    qs = q.shape
    if len(qs) != 4 or q.dtype is not _BF16 or not q.is_contiguous():
        raise ValueError("q: contiguous bf16 [B, T, Hq, D]")
    B, T, Hq, D = qs
    c, _, Hkv, _, width, n_seqs = _pool(k_cache, v_cache, page_table, False)
    index = _same_device(q, k_cache, v_cache, page_table, context_len, draft_len, tree_mask, row_ptr, col_idx, out,
                         lse)
    if n_seqs != B or width != D:
        raise ValueError("page_table needs one row per sequence, the caches q's head size")
    _ints("context_len", context_len, (B,))
    if draft_len is not None:
        _ints("draft_len", draft_len, (B,))
    if tree_mask is not None:
        _ints("tree_mask", tree_mask, (B, T), _I64)
    ci, cap = 0, 0
    if (row_ptr is None) != (col_idx is None):
        raise ValueError("row_ptr and col_idx come together")
    if row_ptr is not None:
        cap = col_idx.numel()
        _ints("row_ptr", row_ptr, (B * Hkv + 1,))
        _ints("col_idx", col_idx, (cap,))
        # an empty list has no storage: any address does, nothing below its capacity of 0 is read
        ci = col_idx.data_ptr() or row_ptr.data_ptr()
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with _scope(index, stream):
        out = _output(out, qs, q)
        if lse is None:
            lse = torch.empty((B, T, Hq), dtype=_F32, device=q.device)
        else:
            _ints("lse", lse, (B, T, Hq), _F32)
        L = lib()
        n = L.bsa_tree_attention_workspace(B, T, Hq, Hkv, D)
        ws = torch.empty(n, dtype=torch.uint8, device=q.device)
        a = _TREE.pack(B, T, Hq, q.data_ptr(), context_len.data_ptr(), _addr(draft_len), _addr(tree_mask),
                       _addr(row_ptr), ci, cap, out.data_ptr(), lse.data_ptr(), scale)
        st = L.bsa_tree_attention(a, c, ws.data_ptr(), n, _raw_stream(index))
    if st:
        _check("bsa_tree_attention", st)
    return out, lse


def cache_accept(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor, context_len: torch.Tensor,
                 accepted: torch.Tensor, n_accepted: torch.Tensor, new_len: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """Moves the rows of the accepted drafts (accepted int32 [n_seqs,T], the
    first n_accepted[b] strictly increasing) up behind the committed slots, in
    every layer of the pools; returns the new lengths context_len + n_accepted."""
    c, _, _, _, _, S = _pool(k_cache, v_cache, page_table, True)
    index = _same_device(k_cache, v_cache, page_table, context_len, accepted, n_accepted, new_len)
    if accepted.dim() != 2:
        raise ValueError("accepted: int32 [n_seqs, T]")
    T = accepted.shape[1]
    _ints("context_len", context_len, (S,))
    _ints("accepted", accepted, (S, T))
    _ints("n_accepted", n_accepted, (S,))
    with _scope(index, stream):
        if new_len is None:
            new_len = torch.empty(S, dtype=_I32, device=context_len.device)
        else:
            _ints("new_len", new_len, (S,))
        st = lib().bsa_cache_accept(c, context_len.data_ptr(), accepted.data_ptr(), n_accepted.data_ptr(), T,
                                    new_len.data_ptr(), _raw_stream(index))
    if st:
        _check("bsa_cache_accept", st)
    return new_len


def _request(fn: str, page_table, page_ref, a, b, n, k_cache, v_cache, stream) -> torch.Tensor:
    c, n_pages, _, _, _, n_seqs = _pool(k_cache, v_cache, page_table, True)
    index = _same_device(k_cache, v_cache, page_table, page_ref, a, b, n)
    _ints("page_ref", page_ref, (n_pages,))
    N = a.numel()
    for t in (a, b, n):
        _ints("requests", t, (N,))
    device = a.device
    with _scope(index, stream):
        granted = torch.empty(N, dtype=_I32, device=device)
        if N == 0:
            return granted
        L = lib()
        size = L.bsa_cache_pages_workspace(N, n_seqs, n_pages)
        ws = torch.empty(size, dtype=torch.uint8, device=device)
        st = getattr(L, fn)(c, page_ref.data_ptr(), N, a.data_ptr(), b.data_ptr(), n.data_ptr(), granted.data_ptr(),
                            ws.data_ptr(), size, _raw_stream(index))
    if st:
        _check(fn, st)
    return granted


def cache_resize(page_table: torch.Tensor, page_ref: torch.Tensor, seqs: torch.Tensor, keep: torch.Tensor,
                 capacity: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, stream=None) -> torch.Tensor:
    """Sequence seqs[i] keeps its first keep[i] slots and holds pages for
    capacity[i] of them (0, 0 frees it); from slot keep[i] on its pages are its
    own.  Updates page_table and page_ref (and copies the kept rows of a shared
    part-filled page); returns int32 1 (served) or 0 (refused) per request."""
    return _request("bsa_cache_resize", page_table, page_ref, seqs, keep, capacity, k_cache, v_cache, stream)


def cache_fork(page_table: torch.Tensor, page_ref: torch.Tensor, src: torch.Tensor, dst: torch.Tensor,
               lens: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, stream=None) -> torch.Tensor:
    """Sequence dst[i] (which holds no page) gets the first lens[i] slots of
    src[i]: full pages shared, the rows of a part-filled last page copied.
    Returns int32 1 (served) or 0 (refused) per request."""
    return _request("bsa_cache_fork", page_table, page_ref, src, dst, lens, k_cache, v_cache, stream)


def cache_compact(page_table: torch.Tensor, page_ref: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  stream=None) -> torch.Tensor:
    """Moves the live pages to the front of the pool, table and counts with
    them; returns int32 [n_pages]: where each page went, -1 for free ones."""
    c, n_pages, _, _, _, n_seqs = _pool(k_cache, v_cache, page_table, True)
    index = _same_device(k_cache, v_cache, page_table, page_ref)
    _ints("page_ref", page_ref, (n_pages,))
    with _scope(index, stream):
        new_page = torch.empty(n_pages, dtype=_I32, device=page_ref.device)
        L = lib()
        size = L.bsa_cache_pages_workspace(0, n_seqs, n_pages)
        ws = torch.empty(size, dtype=torch.uint8, device=page_ref.device)
        st = L.bsa_cache_compact(c, page_ref.data_ptr(), new_page.data_ptr(), ws.data_ptr(), size,
                                 _raw_stream(index))
    if st:
        _check("bsa_cache_compact", st)
    return new_page
