"""The smallest calls of the serving entry points and the edges of their
contracts that the host decides (no GPU needed; the fake pointers are never
dereferenced)."""

import ctypes

import pytest

from test_serving_refusals import FAKE, INVALID, UNSUP, L, cache, rope_args, tree  # noqa: F401


# ------------------------------------------------------------ empty batches
def empty(**kw):
    """What tensors of no sequences give: sizes of 0, null pointers."""
    return cache(**{**dict(n_seqs=0, page_table=None), **kw})


def test_no_sequences_is_nothing_to_do(L):
    t = dict(B=0, q=None, context_len=None, out=None, lse=None)
    assert L.bsa_tree_attention_workspace(0, 4, 8, 2, 128) == 0
    assert L.bsa_tree_attention(ctypes.byref(tree(**t)), ctypes.byref(empty()), None, 0, None) == 0
    lists = dict(row_ptr=FAKE, col_idx=FAKE)
    assert L.bsa_tree_attention(ctypes.byref(tree(**t, **lists)), ctypes.byref(empty()), None, 0, None) == 0
    assert L.bsa_cache_accept(ctypes.byref(empty()), None, None, None, 4, None, None) == 0
    none = rope_args(N=0, q=None, k=None, v=None)
    assert L.bsa_cache_append(ctypes.byref(none), ctypes.byref(empty()), None, None, None, None) == 0
    for fn in (L.bsa_cache_resize, L.bsa_cache_fork):
        assert fn(ctypes.byref(empty()), FAKE, 0, None, None, None, None, None, 0, None) == 0


@pytest.mark.parametrize("bad,st", [(dict(T=0), INVALID), (dict(T=65), UNSUP), (dict(Hq=7), INVALID),
                                    (dict(scale=0.0), INVALID), (dict(B=-1), INVALID), (dict(B=1), INVALID),
                                    (dict(row_ptr=FAKE), INVALID)])
def test_no_sequences_is_still_checked(L, bad, st):
    t = {**dict(B=0, q=None, context_len=None, out=None, lse=None), **bad}
    assert L.bsa_tree_attention(ctypes.byref(tree(**t)), ctypes.byref(empty()), None, 0, None) == st


def test_no_sequences_with_something_to_do(L):
    """Tokens or requests for sequences that there are not, and pools without a table."""
    n = L.bsa_cache_pages_workspace(5, 0, 16)
    c = empty(page_table=FAKE)
    assert L.bsa_cache_append(ctypes.byref(rope_args()), ctypes.byref(c), FAKE, FAKE, FAKE, None) == INVALID
    for fn in (L.bsa_cache_resize, L.bsa_cache_fork):
        assert fn(ctypes.byref(c), FAKE, 5, FAKE, FAKE, FAKE, FAKE, FAKE, n, None) == INVALID
    assert L.bsa_cache_compact(ctypes.byref(c), FAKE, FAKE, FAKE, n, None) == INVALID
    assert L.bsa_cache_accept(ctypes.byref(empty()), None, None, None, 0, None, None) == INVALID
    for kw in (dict(n_seqs=-1), dict(k=None), dict(layers=0), dict(max_pages=0)):
        assert L.bsa_cache_accept(ctypes.byref(empty(**kw)), None, None, None, 4, None, None) == INVALID
    assert L.bsa_cache_accept(ctypes.byref(empty(page=96)), None, None, None, 4, None, None) == UNSUP


# ------------------------------------------------------------ outputs over inputs
def test_accept_refuses_lengths_written_over_what_it_reads(L):
    """Several CTAs read a sequence's entries; one of them writes its new length."""
    c, A, M, N, S = 3 * 4, 1 << 21, 1 << 22, 1 << 23, 1 << 24   # bytes of a vector; addresses

    def accept(new):
        return L.bsa_cache_accept(ctypes.byref(cache(page_table=S)), N, A, M, 4, new, None)

    for base, size in ((N, c), (M, c), (A, 4 * c), (S, 4 * c)):   # lengths, counts, lists, the table
        for at in (base, base + size - 4, base - c + 4):
            assert accept(at) == INVALID, hex(at)


@pytest.mark.parametrize("call", ["bsa_cache_resize", "bsa_cache_fork"])
def test_requests_refuse_answers_written_over_what_they_read(L, call):
    """The last kernel of a request reads the vectors again, after the answers."""
    A, B, C, R, S = (1 << k for k in range(21, 26))
    n = L.bsa_cache_pages_workspace(5, 3, 16)

    def request(granted):
        return getattr(L, call)(ctypes.byref(cache(page_table=S)), R, 5, A, B, C, granted, FAKE, n, None)

    for base, size in ((A, 20), (B, 20), (C, 20), (R, 64), (S, 48)):
        for at in (base, base + size - 4, base - 16):
            assert request(at) == INVALID, hex(at)


def test_compact_refuses_a_map_written_over_what_it_reads(L):
    R, S = 1 << 21, 1 << 22
    n = L.bsa_cache_pages_workspace(0, 3, 16)
    for base, size in ((R, 64), (S, 48)):
        for at in (base, base + size - 4, base - 60):
            assert L.bsa_cache_compact(ctypes.byref(cache(page_table=S)), R, at, FAKE, n, None) == INVALID, hex(at)
