"""Serving over a paged key/value cache: write new tokens, attend with chunks of
them, one or a tree of drafted tokens per sequence, keep the accepted ones, and
the pages.

Pools are bf16 [n_pages, Hkv, page, D] (one layer) or [layers, n_pages, Hkv,
page, D]; a page is a key block of the attention, page in {64, 128}.
page_table is int32 [n_seqs, max_pages] with -1 behind a sequence's pages,
page_ref int32 [n_pages] counts the table entries that hold a page (0: free).

Pools of 8-bit rows are float8_e4m3fn of the same shape, with k_scale and
v_scale, float8_e8m0fnu [(layers,) n_pages, Hkv, page]: a row is its codes times
its scale, a power of two (uint8 tensors of the codes and the scales' bytes
serve too).  Every call here but `tree_attention` takes them.

Marshalling only (``csrc/bsa_torch.cpp``); contracts are in ``include/bsa.h``, the kernels in
``csrc/bsa_rope.cu`` (append), ``csrc/bsa_tree.cu``, ``csrc/bsa_cache.cu``, ``csrc/bsa_chunk.cu``,
``csrc/bsa_decode.cu`` and ``csrc/bsa_read.cu``.
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch

from ._binding import _call, compiled


def cache_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 page_table: torch.Tensor, seq_ids: torch.Tensor, slots: torch.Tensor,
                 inv_freq: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 gain: float = 1.0, interleaved: bool = False, out: Optional[torch.Tensor] = None, stream=None,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None) -> torch.Tensor:
    """`qk_norm_rope` for new tokens of a served batch: token i (q [tokens,Hq,D],
    k, v [tokens,Hkv,D], any strides) belongs to slot slots[i] of sequence
    seq_ids[i] (< 0: padding, skipped), and its rotated key and its value go to
    that slot's page; two tokens of one slot leave pieces of either there.
    positions default to the slots (a tree's drafts give their depth).  8-bit
    pools: keys and values are quantised as they are written, one rounding from
    fp32.  Returns the rotated queries [tokens,Hq,D]."""
    return _call(compiled().cache_append, "bsa_cache_append", stream, q, k, v, inv_freq, positions, q_weight, k_weight,
                 eps, gain, interleaved, 1, k_cache, v_cache, page_table, seq_ids, slots, out, k_scale, v_scale)


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
                 accepted: torch.Tensor, n_accepted: torch.Tensor, new_len: Optional[torch.Tensor] = None, stream=None,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Moves the rows of the accepted drafts (accepted int32 [n_seqs,T], the
    first n_accepted[b] strictly increasing) up behind the committed slots, in
    every layer of the pools; returns the new lengths context_len + n_accepted
    (in new_len, if given: a tensor that overlaps none of the others)."""
    return _call(compiled().cache_accept, "bsa_cache_accept", stream, k_cache, v_cache, page_table, context_len,
                 accepted, n_accepted, new_len, k_scale, v_scale)


def cache_resize(page_table: torch.Tensor, page_ref: torch.Tensor, seqs: torch.Tensor, keep: torch.Tensor,
                 capacity: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, stream=None,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Sequence seqs[i] keeps its first keep[i] slots and holds pages for
    capacity[i] of them (0, 0 frees it); from slot keep[i] on its pages are its
    own.  Updates page_table and page_ref (and copies the kept rows of a shared
    part-filled page); returns int32 1 (served) or 0 (refused) per request."""
    return _call(compiled().cache_request, "bsa_cache_resize", stream, False, page_table, page_ref, seqs, keep,
                 capacity, k_cache, v_cache, k_scale, v_scale)


def cache_fork(page_table: torch.Tensor, page_ref: torch.Tensor, src: torch.Tensor, dst: torch.Tensor,
               lens: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, stream=None,
               k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Sequence dst[i] (which holds no page) gets the first lens[i] slots of
    src[i]: full pages shared, the rows of a part-filled last page copied.
    Returns int32 1 (served) or 0 (refused) per request."""
    return _call(compiled().cache_request, "bsa_cache_fork", stream, True, page_table, page_ref, src, dst, lens,
                 k_cache, v_cache, k_scale, v_scale)


def cache_compact(page_table: torch.Tensor, page_ref: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  stream=None, k_scale: Optional[torch.Tensor] = None,
                  v_scale: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Moves the live pages to the front of the pool, table and counts with
    them; returns int32 [n_pages]: where each page went, -1 for free ones."""
    return _call(compiled().cache_compact, "bsa_cache_compact", stream, page_table, page_ref, k_cache, v_cache, k_scale,
                 v_scale)


def cache_read(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor, seq_ids: torch.Tensor,
               lens: Optional[torch.Tensor], n: int, first: Optional[torch.Tensor] = None, kv_repeat: int = 1,
               k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None, out=None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Slots first[i] .. (default 0) of sequence seq_ids[i] back as what `forward`
    takes: (k, v) bf16 [R, Hkv*kv_repeat, n, D], head h written at h*kv_repeat and
    on.  lens int32 [R] (None: n): rows behind lens[i] are zeros, as are all rows
    of a seq_ids[i] < 0.  out: (k, v) to write."""
    ok, ov = (None, None) if out is None else out
    return _call(compiled().cache_read, "bsa_cache_read", stream, k_cache, v_cache, page_table, seq_ids, lens, n, first,
                 kv_repeat, k_scale, v_scale, ok, ov)


def chunk_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                    context_len: torch.Tensor, q_ptr: Optional[torch.Tensor] = None, window: int = 0, sinks: int = 0,
                    k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                    scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, stream=None,
                    max_context: int = 0) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of new tokens over their sequences' pages: q [tokens,Hq,D] bf16
    (what `cache_append` returns), sequence b's rows q_ptr[b] .. q_ptr[b+1]-1
    (int32 [B+1]; None: one token a sequence) in slots context_len[b] and on.
    Slot s attends to the slots u <= s; with window > 0 only to those with
    u > s - window or u < sinks (pages that no token sees any more may be -1).
    max_context: at least the slots of the longest sequence after this call (0: not
    known, the table's width is taken).  Small batches of chunks and single tokens
    under a wide table are faster with it, and a wrong one gives right results too.

    Weights are rounded to bf16 (2^-8) before they meet V.  Sequences of at most 16
    rows of a key head have finer ones (bf16 pools 2^-16, 8-bit 2^-11) where all are
    such or the batch has work enough for a kernel of their own: a row's last bits
    may depend on the batch and the table's width (the rule is in ``include/bsa.h``).

    Returns (O bf16 [tokens,Hq,D], LSE fp32 [tokens,Hq]); rows of no sequence
    are left as they were."""
    return _call(compiled().chunk_attention, "bsa_chunk_attention", stream, q, k_cache, v_cache, page_table,
                 context_len, q_ptr, window, sinks, k_scale, v_scale, scale, out, lse, max_context)
