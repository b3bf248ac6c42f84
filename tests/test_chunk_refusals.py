"""Refusals of the chunk attention, of reading a cache back and of the 8-bit cache's
calls: every call here returns before it touches a device (no GPU needed; the
fake pointers are never dereferenced)."""

import ctypes
import math

import pytest
import torch

from test_serving_refusals import FAKE, INVALID, UNSUP, CAPACITY, L, cache, rope_args  # noqa: F401


def scales(**kw):
    from block_sparse_flashattention_bsa_gb300._binding import _PageScales
    return _PageScales(**{**dict(k=FAKE, v=FAKE), **kw})


def chunk(**kw):
    from block_sparse_flashattention_bsa_gb300._binding import _ChunkArgs
    a = dict(B=3, tokens=40, Hq=8, q=FAKE, q_ptr=FAKE, context_len=FAKE, out=FAKE, lse=FAKE, scale=0.1, window=0, sinks=0)
    a.update(kw)
    return _ChunkArgs(**a)


def read(**kw):
    from block_sparse_flashattention_bsa_gb300._binding import _ReadArgs
    a = dict(R=2, n=100, kv_repeat=1, seq_ids=FAKE, first=None, len=FAKE, k=FAKE, v=FAKE)
    a.update(kw)
    return _ReadArgs(**a)


ref = ctypes.byref
WS = 1 << 28


@pytest.mark.parametrize("bad,st", [
    (dict(B=-1), INVALID), (dict(tokens=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hq=7), INVALID),
    (dict(Hq=2 * 129), UNSUP), (dict(B=2), INVALID), (dict(q=None), INVALID), (dict(context_len=None), INVALID),
    (dict(out=None), INVALID), (dict(lse=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(out=FAKE + 8), INVALID),
    (dict(lse=FAKE + 2), INVALID), (dict(context_len=FAKE + 1), INVALID), (dict(q_ptr=FAKE + 2), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID),
    (dict(scale=math.inf), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(q_ptr=None), INVALID),
    (dict(tokens=2 ** 31 - 1, Hq=256), INVALID)], ids=lambda x: str(x))
@pytest.mark.parametrize("q8", [False, True])
def test_chunk_attention_refuses(L, bad, st, q8):
    s = ref(scales()) if q8 else None
    c = cache(max_pages=1 << 16) if bad.get("tokens", 0) > 40 else cache()
    assert L.bsa_chunk_attention(ref(chunk(**bad)), ref(c), s, FAKE, WS, None) == st


@pytest.mark.parametrize("bad,st", [(dict(layers=2), INVALID), (dict(page=32), UNSUP), (dict(D=96), UNSUP),
                                    (dict(k=None), INVALID), (dict(v=FAKE + 8), INVALID), (dict(page_table=None), INVALID),
                                    (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID)], ids=lambda x: str(x))
def test_chunk_attention_refuses_caches(L, bad, st):
    assert L.bsa_chunk_attention(ref(chunk()), ref(cache(**bad)), None, FAKE, WS, None) == st


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 1)])
def test_scales_are_checked(L, bad):
    c, s = cache(), scales(**bad)
    assert L.bsa_chunk_attention(ref(chunk()), ref(c), ref(s), FAKE, WS, None) == INVALID
    assert L.bsa_cache_read(ref(read()), ref(c), ref(s), None) == INVALID
    assert L.bsa_cache_append_fp8(ref(rope_args()), ref(c), ref(s), FAKE, FAKE, FAKE, None) == INVALID
    assert L.bsa_cache_resize_fp8(ref(c), ref(s), FAKE, 1, FAKE, FAKE, FAKE, FAKE, FAKE, WS, None) == INVALID
    assert L.bsa_cache_fork_fp8(ref(c), ref(s), FAKE, 1, FAKE, FAKE, FAKE, FAKE, FAKE, WS, None) == INVALID
    assert L.bsa_cache_compact_fp8(ref(c), ref(s), FAKE, FAKE, FAKE, WS, None) == INVALID
    assert L.bsa_cache_accept_fp8(ref(c), ref(s), FAKE, FAKE, FAKE, 4, FAKE, None) == INVALID


def test_fp8_calls_need_scales_and_check_the_rest(L):
    c, s = cache(), scales()
    assert L.bsa_cache_append_fp8(ref(rope_args()), ref(c), None, FAKE, FAKE, FAKE, None) == INVALID
    assert L.bsa_cache_resize_fp8(ref(c), None, FAKE, 1, FAKE, FAKE, FAKE, FAKE, FAKE, WS, None) == INVALID
    assert L.bsa_cache_fork_fp8(ref(c), None, FAKE, 1, FAKE, FAKE, FAKE, FAKE, FAKE, WS, None) == INVALID
    assert L.bsa_cache_compact_fp8(ref(c), None, FAKE, FAKE, FAKE, WS, None) == INVALID
    assert L.bsa_cache_accept_fp8(ref(c), None, FAKE, FAKE, FAKE, 4, FAKE, None) == INVALID
    # what their namesakes refuse
    assert L.bsa_cache_append_fp8(ref(rope_args(eps=-1.0)), ref(c), ref(s), FAKE, FAKE, FAKE, None) == INVALID
    assert L.bsa_cache_append_fp8(ref(rope_args()), ref(cache(D=64)), ref(s), FAKE, FAKE, FAKE, None) == INVALID
    assert L.bsa_cache_append_fp8(ref(rope_args()), ref(c), ref(s), FAKE, FAKE, None, None) == INVALID
    assert L.bsa_cache_resize_fp8(ref(c), ref(s), FAKE, -1, FAKE, FAKE, FAKE, FAKE, FAKE, WS, None) == INVALID
    assert L.bsa_cache_fork_fp8(ref(c), ref(s), FAKE, 1, FAKE, FAKE, FAKE, FAKE, FAKE, 16, None) == CAPACITY
    assert L.bsa_cache_compact_fp8(ref(c), ref(s), FAKE, FAKE, FAKE, 16, None) == CAPACITY
    assert L.bsa_cache_accept_fp8(ref(c), ref(s), FAKE, FAKE, FAKE, 65, FAKE, None) == INVALID


def test_workspace(L):
    n = L.bsa_chunk_attention_workspace(3, 40, 8, 2, 128)
    assert n > 0 and L.bsa_chunk_attention_workspace(3, 3, 8, 2, 128) < n
    assert L.bsa_chunk_attention(ref(chunk()), ref(cache()), None, FAKE, n - 1, None) == CAPACITY
    assert L.bsa_chunk_attention(ref(chunk()), ref(cache()), None, None, n, None) == INVALID
    assert L.bsa_chunk_attention(ref(chunk()), ref(cache()), None, FAKE + 128, n, None) == INVALID
    for bad in ((0, 4, 8, 2, 128), (3, 0, 8, 2, 128), (3, 4, 7, 2, 128), (3, 4, 8, 0, 128), (3, 4, 8, 2, 0), (3, 4, 258, 2, 128)):
        assert L.bsa_chunk_attention_workspace(*bad) == 0


def test_nothing_to_do(L):
    none = dict(q=None, context_len=None, out=None, lse=None, q_ptr=None)
    empty = cache(n_seqs=0, page_table=None)
    assert L.bsa_chunk_attention(ref(chunk(B=0, tokens=0, **none)), ref(empty), None, None, 0, None) == 0
    assert L.bsa_chunk_attention(ref(chunk(tokens=0)), ref(cache()), None, None, 0, None) == 0
    assert L.bsa_chunk_attention(ref(chunk(B=0, tokens=0, scale=0.0, **none)), ref(empty), None, None, 0, None) == INVALID
    assert L.bsa_cache_read(ref(read(R=0)), ref(empty), None, None) == 0
    assert L.bsa_cache_read(ref(read(n=0)), ref(cache()), None, None) == 0
    assert L.bsa_cache_append_fp8(ref(rope_args(N=0, q=None, k=None, v=None)), ref(empty), ref(scales()), None, None, None,
                                  None) == 0
    assert L.bsa_cache_accept_fp8(ref(empty), ref(scales()), None, None, None, 4, None, None) == 0


@pytest.mark.parametrize("bad", [dict(R=-1), dict(n=-1), dict(kv_repeat=0), dict(seq_ids=None), dict(k=None), dict(v=None),
                                 dict(k=FAKE + 8), dict(v=FAKE + 4), dict(seq_ids=FAKE + 2), dict(first=FAKE + 1),
                                 dict(len=FAKE + 3), dict(kv_repeat=1 << 30),
                                 dict(R=2 ** 31 - 1, n=2 ** 31 - 1, kv_repeat=1 << 20)], ids=lambda b: "-".join(b))
def test_cache_read_refuses(L, bad):
    assert L.bsa_cache_read(ref(read(**bad)), ref(cache()), None, None) == INVALID


def test_cache_read_refuses_caches(L):
    assert L.bsa_cache_read(None, ref(cache()), None, None) == INVALID
    assert L.bsa_cache_read(ref(read()), None, None, None) == INVALID
    assert L.bsa_cache_read(ref(read()), ref(cache(layers=2)), None, None) == INVALID
    assert L.bsa_cache_read(ref(read()), ref(cache(n_seqs=0)), None, None) == INVALID
    assert L.bsa_cache_read(ref(read()), ref(cache(D=80)), None, None) == UNSUP


# ------------------------------------------------------------ the Python layer, on CPU tensors
def pools(q8=False, D=64):
    t = torch.zeros(4, 2, 64, D, dtype=torch.float8_e4m3fn if q8 else torch.bfloat16)
    return t, t.clone(), torch.zeros(1, 3, dtype=torch.int32)


def test_python_checks():
    import block_sparse_flashattention_bsa_gb300 as bsa
    i = torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    k, v, table = pools()
    s = torch.zeros(4, 2, 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        bsa.chunk_attention(q, k, v, table, i)
    with pytest.raises(ValueError, match="together"):
        bsa.chunk_attention(q, k, v, table, i, k_scale=s)
    with pytest.raises(ValueError, match="e4m3"):
        bsa.chunk_attention(q, k, v, table, i, k_scale=s, v_scale=s)
    k8, v8, _ = pools(True)
    with pytest.raises(ValueError, match="bf16"):
        bsa.chunk_attention(q, k8, v8, table, i)
    for bad in (s[:, :, :32], s.float(), s.transpose(1, 2)):
        with pytest.raises(ValueError, match="e8m0"):
            bsa.chunk_attention(q, k8, v8, table, i, k_scale=bad, v_scale=bad)
    with pytest.raises(ValueError, match="q:"):
        bsa.chunk_attention(q.float(), k, v, table, i)
    with pytest.raises(ValueError):
        bsa.cache_read(k, v, table.float(), i, None, 8)
    with pytest.raises(ValueError, match="tensor"):
        bsa.cache_read(k, v, table, None, None, 8)
    with pytest.raises(ValueError, match="bf16"):
        bsa.tree_attention(q[None], k8, v8, table, i)
