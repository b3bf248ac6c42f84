"""Refusals of the projection, paged-cache and tree-attention entry points:
every call here returns before it touches a device (no GPU needed; the fake
pointers are never dereferenced), and the frequencies, which are host code."""

import ctypes
import math

import numpy as np
import pytest
import torch

INVALID, UNSUP, CAPACITY = -1, -2, -3
P = ctypes.c_void_p
FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    from block_sparse_flashattention_bsa_gb300 import build as B
    B.build()
    import block_sparse_flashattention_bsa_gb300 as bsa
    return bsa.lib()


def rope_args(**kw):
    from block_sparse_flashattention_bsa_gb300._binding import _NormRopeArgs, _Stride3
    a = dict(B=1, N=8, Hq=4, Hkv=2, D=128, rotary_dim=64, kv_repeat=1, interleaved=0, eps=1e-6, gain=1.0, q=FAKE,
             k=FAKE, v=FAKE, q_stride=_Stride3(8192, 1024, 128), k_stride=_Stride3(8192, 1024, 128),
             v_stride=_Stride3(8192, 1024, 128), inv_freq=FAKE, positions=None, position_stride=0, q_weight=FAKE,
             k_weight=FAKE)
    a.update(kw)
    return _NormRopeArgs(**a)


def cache(**kw):
    from block_sparse_flashattention_bsa_gb300._binding import _PageCache
    c = dict(k=FAKE, v=FAKE, layers=1, n_pages=16, Hkv=2, page=128, D=128, page_table=FAKE, n_seqs=3, max_pages=4)
    c.update(kw)
    return _PageCache(**c)


BAD_SIDES = [dict(B=-1), dict(N=-1), dict(Hq=0), dict(Hkv=0), dict(kv_repeat=0), dict(rotary_dim=24),
             dict(rotary_dim=144), dict(rotary_dim=-16), dict(interleaved=2), dict(eps=-1.0), dict(eps=math.nan),
             dict(gain=math.inf), dict(inv_freq=None), dict(q=FAKE + 8), dict(k=FAKE + 2), dict(v=FAKE + 4),
             dict(q_stride=(ctypes.c_int64 * 3)(8192, 1020, 128)), dict(k_stride=(ctypes.c_int64 * 3)(-8, 8, 8)),
             dict(positions=FAKE + 2), dict(position_stride=-1), dict(B=1 << 20, N=1 << 20), dict(q=None),
             dict(k=None), dict(kv_repeat=1 << 30)]


@pytest.mark.parametrize("bad", BAD_SIDES, ids=lambda b: "-".join(b))
def test_norm_rope_refuses(L, bad):
    assert L.bsa_qk_norm_rope(ctypes.byref(rope_args(**bad)), FAKE, FAKE, FAKE, None) == INVALID


def test_norm_rope_refuses_outputs_and_head_size(L):
    a = rope_args()
    assert L.bsa_qk_norm_rope(None, FAKE, FAKE, FAKE, None) == INVALID
    assert L.bsa_qk_norm_rope(ctypes.byref(a), None, FAKE, FAKE, None) == INVALID
    assert L.bsa_qk_norm_rope(ctypes.byref(a), FAKE, FAKE, None, None) == INVALID       # v without v_out
    assert L.bsa_qk_norm_rope(ctypes.byref(a), FAKE, FAKE + 8, FAKE, None) == INVALID
    assert L.bsa_qk_norm_rope(ctypes.byref(rope_args(v=None)), FAKE, FAKE, FAKE, None) == INVALID
    assert L.bsa_qk_norm_rope(ctypes.byref(rope_args(D=96)), FAKE, FAKE, FAKE, None) == UNSUP
    # nothing to do: no tokens
    assert L.bsa_qk_norm_rope(ctypes.byref(rope_args(N=0, q=None, k=None, v=None)), None, None, None, None) == 0


def grads(**kw):
    from block_sparse_flashattention_bsa_gb300._binding import _NormRopeGrads, _Stride3
    g = dict(dq=FAKE, dk=FAKE, dv=FAKE, q=FAKE, k=FAKE, v=FAKE, q_stride=_Stride3(8192, 1024, 128),
             k_stride=_Stride3(8192, 1024, 128), v_stride=_Stride3(8192, 1024, 128), q_weight=FAKE, k_weight=FAKE)
    g.update(kw)
    return _NormRopeGrads(**g)


def test_norm_rope_backward_refuses(L):
    n = L.bsa_qk_norm_rope_backward_workspace(128)
    assert n > 0

    def call(a=None, g=None, ws=FAKE, size=n):
        return L.bsa_qk_norm_rope_backward(ctypes.byref(a or rope_args()), ctypes.byref(g or grads()), ws, size, None)

    assert call(g=grads(dq=None)) == INVALID
    assert call(g=grads(dv=None)) == INVALID                                # a gradient of v without dv
    assert call(g=grads(q=FAKE + 8)) == INVALID
    assert call(g=grads(q_weight=None)) == INVALID                          # weight without its gradient
    assert call(a=rope_args(q_weight=None)) == INVALID                      # gradient without its weight
    assert call(g=grads(k_weight=FAKE + 4)) == INVALID
    assert call(g=grads(k_stride=(ctypes.c_int64 * 3)(0, 0, 128))) == INVALID   # rows would coincide
    assert call(a=rope_args(q=None)) == INVALID
    assert call(ws=None) == CAPACITY and call(size=n - 1) == CAPACITY
    assert call(ws=FAKE + 4) == INVALID


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=FAKE + 8), dict(n_pages=0), dict(n_seqs=0), dict(max_pages=0),
                                 dict(layers=0), dict(layers=2), dict(Hkv=3), dict(page_table=None),
                                 dict(page_table=FAKE + 2), dict(n_pages=1 << 24), dict(max_pages=1 << 25)],
                         ids=lambda b: "-".join(b))
def test_append_refuses_caches(L, bad):
    assert L.bsa_cache_append(ctypes.byref(rope_args()), ctypes.byref(cache(**bad)), FAKE, FAKE, FAKE, None) == INVALID


def test_append_refuses(L):
    def call(a=None, c=None, seq=FAKE, slot=FAKE, out=FAKE):
        return L.bsa_cache_append(ctypes.byref(a or rope_args()), ctypes.byref(c or cache()), seq, slot, out, None)

    assert call(a=rope_args(B=2)) == INVALID and call(a=rope_args(kv_repeat=2)) == INVALID
    assert call(seq=None) == INVALID and call(slot=FAKE + 2) == INVALID and call(out=FAKE + 8) == INVALID
    assert call(a=rope_args(v=None)) == INVALID
    assert call(c=cache(page=96)) == UNSUP and call(c=cache(D=256)) == UNSUP
    assert call(c=cache(D=64)) == INVALID                                   # not the rows' head size


def tree(**kw):
    from block_sparse_flashattention_bsa_gb300._binding import _TreeArgs
    a = dict(B=3, T=4, Hq=8, q=FAKE, context_len=FAKE, draft_len=None, tree_mask=None, row_ptr=None, col_idx=None,
             col_capacity=0, out=FAKE, lse=FAKE, scale=0.1)
    a.update(kw)
    return _TreeArgs(**a)


@pytest.mark.parametrize("bad,st", [(dict(B=2), INVALID), (dict(T=0), INVALID), (dict(T=65), UNSUP),
                                    (dict(Hq=7), INVALID), (dict(Hq=2 * 129), UNSUP), (dict(q=None), INVALID),
                                    (dict(q=FAKE + 8), INVALID), (dict(out=FAKE + 2), INVALID),
                                    (dict(lse=None), INVALID), (dict(context_len=None), INVALID),
                                    (dict(tree_mask=FAKE + 4), INVALID), (dict(row_ptr=FAKE), INVALID),
                                    (dict(row_ptr=FAKE, col_idx=FAKE, col_capacity=-1), INVALID),
                                    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
                                    (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID)])
def test_tree_refuses(L, bad, st):
    big = 1 << 40
    assert L.bsa_tree_attention(ctypes.byref(tree(**bad)), ctypes.byref(cache()), FAKE, big, None) == st


def test_tree_refuses_workspaces(L):
    n = L.bsa_tree_attention_workspace(3, 4, 8, 2, 128)
    assert n > 0 and L.bsa_tree_attention_workspace(3, 4, 7, 2, 128) == 0
    a, c = tree(), cache()
    assert L.bsa_tree_attention(ctypes.byref(a), ctypes.byref(c), None, n, None) == INVALID
    assert L.bsa_tree_attention(ctypes.byref(a), ctypes.byref(c), FAKE + 128, n, None) == INVALID
    assert L.bsa_tree_attention(ctypes.byref(a), ctypes.byref(c), FAKE, n - 1, None) == CAPACITY
    assert L.bsa_tree_attention(ctypes.byref(a), ctypes.byref(cache(layers=2)), FAKE, n, None) == INVALID


def test_accept_and_pages_refuse(L):
    c = cache()

    def accept(T=4, new=FAKE + 64, acc=FAKE):
        return L.bsa_cache_accept(ctypes.byref(c), FAKE, acc, FAKE, T, new, None)

    assert accept(T=0) == INVALID and accept(T=65) == INVALID and accept(acc=None) == INVALID
    assert accept(new=FAKE) == INVALID                                      # new_len is context_len
    n = L.bsa_cache_pages_workspace(5, 3, 16)
    for fn in (L.bsa_cache_resize, L.bsa_cache_fork):
        assert fn(ctypes.byref(c), FAKE, -1, FAKE, FAKE, FAKE, FAKE, FAKE, n, None) == INVALID
        assert fn(ctypes.byref(c), FAKE, 0, None, None, None, None, None, 0, None) == 0
        assert fn(ctypes.byref(c), None, 5, FAKE, FAKE, FAKE, FAKE, FAKE, n, None) == INVALID
        assert fn(ctypes.byref(c), FAKE, 5, FAKE, FAKE, FAKE + 1, FAKE, FAKE, n, None) == INVALID
        assert fn(ctypes.byref(c), FAKE, 5, FAKE, FAKE, FAKE, FAKE, FAKE, n - 1, None) == CAPACITY
        assert fn(ctypes.byref(c), FAKE, 5, FAKE, FAKE, FAKE, FAKE, FAKE + 4, n, None) == INVALID
    assert L.bsa_cache_compact(ctypes.byref(c), None, FAKE, FAKE, n, None) == INVALID
    assert L.bsa_cache_compact(ctypes.byref(c), FAKE, FAKE, FAKE, 8, None) == CAPACITY


def test_binding_refuses_wrong_tensors(L):
    import block_sparse_flashattention_bsa_gb300 as bsa
    x = torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16)
    f = torch.zeros(32, dtype=torch.float64)
    kc = torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16)
    tab, one = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    ref = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: bsa.qk_norm_rope(x, x, x, f), lambda: bsa.qk_norm_rope_backward(x, x, x, x, x, f),
                 lambda: bsa.tree_attention(x, kc, kc, tab, one), lambda: bsa.cache_compact(tab, ref, kc, kc),
                 lambda: bsa.cache_accept(kc, kc, tab, one, tab, one),
                 lambda: bsa.cache_append(x[0], x[0], x[0], kc, kc, tab, one, one, f),
                 lambda: bsa.cache_resize(tab, ref, one, one, one, kc, kc),
                 lambda: bsa.cache_fork(tab, ref, one, one, one, kc, kc),
                 lambda: bsa.rope_inv_freq(64, scaling="other")):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------ frequencies
def test_inv_freq_values(L):
    import block_sparse_flashattention_bsa_gb300 as bsa
    i = np.arange(32)
    plain = 500000.0 ** (-2 * i / 64)
    got = bsa.rope_inv_freq(64, 500000.0, device="cpu").numpy()
    np.testing.assert_allclose(got, plain, rtol=1e-14)  # a few roundings of 2^-53
    np.testing.assert_allclose(bsa.rope_inv_freq(64, 500000.0, "linear", 4.0, device="cpu").numpy(), plain / 4,
                               rtol=1e-14)
    b = (500000.0 * 4.0 ** (64 / 62)) ** (-2 * i / 64)
    np.testing.assert_allclose(bsa.rope_inv_freq(64, 500000.0, "base", 4.0, device="cpu").numpy(), b, rtol=1e-13)
    parts = bsa.rope_inv_freq(64, 500000.0, "by_parts", 8.0, original_length=8192, low=1, high=4,
                              device="cpu").numpy()
    turns = 8192 * plain / (2 * np.pi)
    ramp = np.clip((turns - 1) / 3, 0, 1)
    np.testing.assert_allclose(parts, plain * (ramp + (1 - ramp) / 8), rtol=1e-13)
    assert parts[0] == got[0] and abs(parts[-1] * 8 / got[-1] - 1) < 1e-14


@pytest.mark.parametrize("bad", [dict(rotary_dim=0), dict(rotary_dim=63), dict(base=0.0), dict(base=math.inf),
                                 dict(scaling="linear", factor=0.0), dict(scaling="base", rotary_dim=2),
                                 dict(scaling="by_parts"),
                                 dict(scaling="by_parts", original_length=8192, low=4, high=4)], ids=str)
def test_inv_freq_refuses(L, bad):
    import block_sparse_flashattention_bsa_gb300 as bsa
    with pytest.raises(bsa.BsaError):
        bsa.rope_inv_freq(**{**dict(rotary_dim=64, device="cpu"), **bad})
