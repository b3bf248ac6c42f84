"""Serving over a paged key/value cache: write new tokens, attend with one or
a tree of drafted tokens per sequence, keep the accepted ones, and the pages.

Pools are bf16 [n_pages, Hkv, page, D] (one layer) or [layers, n_pages, Hkv,
page, D]; a page is a key block of the attention, page in {64, 128}.
page_table is int32 [n_seqs, max_pages] with -1 behind a sequence's pages,
page_ref int32 [n_pages] counts the table entries that hold a page (0: free).

Marshalling only (``csrc/bsa_torch.cpp``); contracts are in ``include/bsa.h``, the kernels in
``csrc/bsa_rope.cu`` (append), ``csrc/bsa_tree.cu`` and ``csrc/bsa_cache.cu``.
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch

from ._binding import _call, compiled


def cache_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 page_table: torch.Tensor, seq_ids: torch.Tensor, slots: torch.Tensor,
                 inv_freq: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 gain: float = 1.0, interleaved: bool = False, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """`qk_norm_rope` for new tokens of a served batch: token i (q [tokens,Hq,D],
    k, v [tokens,Hkv,D], any strides) belongs to slot slots[i] of sequence
    seq_ids[i] (< 0: padding, skipped), and its rotated key and its value go to
    that slot's page; two tokens of one slot leave pieces of either there.
    positions default to the slots (a tree's drafts give their depth).  Returns
    the rotated queries [tokens,Hq,D]."""
    return _call(compiled().cache_append, "bsa_cache_append", stream, q, k, v, inv_freq, positions, q_weight, k_weight,
                 eps, gain, interleaved, 1, k_cache, v_cache, page_table, seq_ids, slots, out)


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
    return _call(compiled().tree_attention, "bsa_tree_attention", stream, q, k_cache, v_cache, page_table, context_len,
                 draft_len, tree_mask, row_ptr, col_idx, scale, out, lse)


def cache_accept(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor, context_len: torch.Tensor,
                 accepted: torch.Tensor, n_accepted: torch.Tensor, new_len: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """Moves the rows of the accepted drafts (accepted int32 [n_seqs,T], the
    first n_accepted[b] strictly increasing) up behind the committed slots, in
    every layer of the pools; returns the new lengths context_len + n_accepted
    (in new_len, if given: a tensor that overlaps none of the others)."""
    return _call(compiled().cache_accept, "bsa_cache_accept", stream, k_cache, v_cache, page_table, context_len,
                 accepted, n_accepted, new_len)


def cache_resize(page_table: torch.Tensor, page_ref: torch.Tensor, seqs: torch.Tensor, keep: torch.Tensor,
                 capacity: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, stream=None) -> torch.Tensor:
    """Sequence seqs[i] keeps its first keep[i] slots and holds pages for
    capacity[i] of them (0, 0 frees it); from slot keep[i] on its pages are its
    own.  Updates page_table and page_ref (and copies the kept rows of a shared
    part-filled page); returns int32 1 (served) or 0 (refused) per request."""
    return _call(compiled().cache_request, "bsa_cache_resize", stream, False, page_table, page_ref, seqs, keep,
                 capacity, k_cache, v_cache)


def cache_fork(page_table: torch.Tensor, page_ref: torch.Tensor, src: torch.Tensor, dst: torch.Tensor,
               lens: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, stream=None) -> torch.Tensor:
    """Sequence dst[i] (which holds no page) gets the first lens[i] slots of
    src[i]: full pages shared, the rows of a part-filled last page copied.
    Returns int32 1 (served) or 0 (refused) per request."""
    return _call(compiled().cache_request, "bsa_cache_fork", stream, True, page_table, page_ref, src, dst, lens,
                 k_cache, v_cache)


def cache_compact(page_table: torch.Tensor, page_ref: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  stream=None) -> torch.Tensor:
    """Moves the live pages to the front of the pool, table and counts with
    them; returns int32 [n_pages]: where each page went, -1 for free ones."""
    return _call(compiled().cache_compact, "bsa_cache_compact", stream, page_table, page_ref, k_cache, v_cache)
