"""The weights' gradients of qk_norm_rope_backward: a bound close enough that a lost
token shows, which is shown on the CPU (planted in the 64-bit reference).

A sum over rows of t = dy * x * r.  A term's errors: cos and
sin are off by 2^-20, and |dz_a| + |dz_b| is at most sqrt 2 times the pair's
length: 2^-19 of the length; r by 2^-22 and half of the 20 additions behind it,
2^-20; roundings and the sum of up to eight copies 2^-19: together below 2^-17
of (length of dy's pair) * |x| r.  The sum: 2^-24 of sum |t| per addition along
the longest chain: the rows of a lane, at most three times an even share of
rows / (SMs * lane groups) (a kind gets at least half a CTA per SM, tasks are
uneven by less than 1.5), then 3 levels in a warp, 8 warps, at most 19 CTAs per
thread of the last kernel and its 6 levels: 36, and single rows of small calls:
64 covers them.  A token that is left out (all heads of it) is off by more than
that in some column."""

import numpy as np
import pytest
import torch

from test_gpu_rope import dev, f64, make


@pytest.fixture(scope="module")
def bsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_flashattention_bsa_gb300 import build
    build.build()
    import block_sparse_flashattention_bsa_gb300 as m
    m.device_error()
    return m


GRADS = [  # B, N, Hq, Hkv, rep, D, rd, interleaved, norm, positions; the last three with four CTAs per SM
    (1, 1000, 16, 4, 1, 128, 64, False, "qk", None),
    (2, 515, 7, 1, 7, 64, 16, False, "qk", None),
    (1, 4099, 20, 5, 4, 64, 64, True, "qk", "row"),
    (2, 127, 6, 3, 2, 64, 48, True, "k", "negative"),
    (1, 8229, 16, 16, 1, 128, 128, False, "qk", "row"),
    (1, 17011, 20, 5, 4, 64, 32, True, "qk", None),
    (3, 4099, 13, 13, 1, 128, 112, False, "q", "batch"),
]
SMS = 152


def weight_terms(x, dz, pos, freq, eps, gain, il, D):
    """Rows' contributions dy * x * r [rows, D] and the length of dy's pairs times |x| r."""
    dy, size = dz.copy(), np.abs(dz)
    if freq is not None:
        rd, i = 2 * len(freq), np.arange(len(freq))
        a, b = (2 * i, 2 * i + 1) if il else (i, i + rd // 2)
        ang = pos[..., None].astype(np.float64) * freq
        c, s = np.cos(ang)[..., None, :], np.sin(ang)[..., None, :]
        dy[..., a] = gain * (dz[..., a] * c + dz[..., b] * s)
        dy[..., b] = gain * (dz[..., b] * c - dz[..., a] * s)
        size[..., a] = size[..., b] = np.hypot(dy[..., a], dy[..., b])
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return (dy * x * r).reshape(-1, D), (size * np.abs(x) * r).reshape(-1, D)


def bound_of(t, size, rows, D):
    chain = 3 * -(-rows // (SMS * 256 * 16 // D)) + 64
    return size.sum(0) * 2.0 ** -17 + np.abs(t).sum(0) * chain * 2.0 ** -24


def inputs(case):
    B, N, Hq, Hkv, rep, D, rd, il, norm, how = case
    g = torch.Generator().manual_seed(11)
    return make(case, 90), [torch.randn(B, H, N, D, generator=g).bfloat16() for H in (Hq, Hkv * rep, Hkv * rep)]


def sides(case, qkv, dz, p, freq):
    """(terms, sizes) of q and k, [B N H, D] in the order of the tokens; None without a weight."""
    B, N, Hq, Hkv, rep, D, rd, il, norm, how = case
    X, fr = f64(qkv), freq.numpy()
    for name, lo, hi, r, d in (("q", 0, Hq, 1, dz[0]), ("k", Hq, Hq + Hkv, rep, dz[1])):
        if name not in norm:
            yield None
            continue
        d = f64(d).reshape(B, hi - lo, r, N, D).sum(2).transpose(0, 2, 1, 3)
        yield weight_terms(X[:, :, lo:hi], d, p, fr, 1e-5, 0.75, il, D)


@pytest.mark.parametrize("case", GRADS, ids=str)
def test_the_bound_sees_a_lost_token(case):
    (qkv, qw, kw, freq, pos, p), dz = inputs(case)
    for side in sides(case, qkv, dz, p, freq):
        if side is not None:
            t, size = side
            token = t.reshape(case[0] * case[1], -1, case[5]).sum(1)
            seen = (np.abs(token) > bound_of(t, size, len(t), case[5])).any(-1)
            assert seen[-1] and seen.mean() >= 0.95


@pytest.mark.gpu
@pytest.mark.parametrize("case", GRADS, ids=str)
def test_weight_gradients(bsa, case):
    B, N, Hq, Hkv, rep, D, rd, il, norm, how = case
    assert torch.cuda.get_device_properties(0).multi_processor_count == SMS
    (qkv, qw, kw, freq, pos, p), dz = inputs(case)
    x, dqw, dkw, dfreq, dpos, *ddz = dev(qkv, qw, kw, freq, pos, *dz)
    got = bsa.qk_norm_rope_backward(*ddz, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], dfreq, positions=dpos, q_weight=dqw,
                                    k_weight=dkw, eps=1e-5, gain=0.75, interleaved=il, kv_repeat=rep)[3:]
    for gw, side in zip(got, sides(case, qkv, dz, p, freq)):
        assert (gw is None) == (side is None)
        if side is not None:
            t, size = side
            assert (np.abs(f64(gw) - t.sum(0)) <= bound_of(t, size, len(t), D)).all()
    assert bsa.device_error() == 0
