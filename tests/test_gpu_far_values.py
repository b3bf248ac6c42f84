"""Single tokens over caches whose values' magnitudes lie far apart while the
scores' maxima grow: what is met first, with next to no weight, drowns nothing
that follows.

Tolerances are test_gpu_chunk's: weights to 2^-11 (8-bit rows: weight times scale,
rounded to fp16 once) or 2^-16 (bf16 rows), of A = sum p |v| / sum p.  M, the scores'
part of them, is at most 110 here: with D = 128 that is 2 e <= 2^-9 of A, far below
what a lost row takes from O.
"""


import pytest
import torch

from paged_reference import Cache, attention, check_attention, quantise
from test_gpu_chunk import both, bsa  # noqa: F401

pytestmark = pytest.mark.gpu

N = 2560            # slots of a sequence
LOG2E = 1.4426950408889634


def steep_cache(D, Hkv, B, q8, score, size, seed):
    """B sequences of the same N slots: keys whose first value makes score(slot) (log2, times the query's
    first value) of the score, values of magnitude 2^size(slot) (lists, per slot)."""
    g = torch.Generator().manual_seed(seed)
    c = Cache([1] * B, Hkv, D, 64, q8, seed)
    P = N // 64
    c.n_pages = P + 1
    order = torch.randperm(P, generator=g).int()
    c.table = torch.cat([order, order.new_full((1,), -1)]).expand(B, -1).contiguous()
    k = torch.randn(Hkv, N, D, generator=g, dtype=torch.float64) * 0.05
    k[..., 0] = torch.tensor(score, dtype=torch.float64) / LOG2E * D ** 0.5
    v = torch.randn(Hkv, N, D, generator=g, dtype=torch.float64) * torch.pow(2.0, torch.tensor(size, dtype=torch.float64))[:, None]
    for name, x in zip("kv", (k, v)):
        pages = torch.empty(P + 1, Hkv, 64, D, dtype=torch.float64)
        pages[order.long()] = x.reshape(Hkv, P, 64, D).transpose(0, 1)
        pages[P] = 0
        if q8:
            codes, scales = quantise(pages)
            setattr(c, name, codes)
            setattr(c, name + "s", scales)
        else:
            setattr(c, name, pages.bfloat16())
    return c


def check(bsa, c, q, q8):  # noqa: F811
    B, D = q.shape[0], q.shape[2]
    k, v, table, sc = c.device()
    ctx = torch.full((B,), N - 1, dtype=torch.int32)
    o, lse = bsa.chunk_attention(q.cuda(), k, v, table.cuda(), ctx.cuda(), **sc)
    assert bsa.device_error() == 0
    ref = attention(c, q, list(range(B + 1)), ctx.tolist(), 0, 0, D ** -0.5)
    check_attention(o, lse, ref, D, 2.0 ** -11 if q8 else 2.0 ** -16)
    return o, lse


def queries(B, Hq, D, first, seed):
    q = torch.randn(B, Hq, D, generator=torch.Generator().manual_seed(seed)) * 0.2
    q[..., 0] = first
    return q.bfloat16()


# B, Hkv, G: a CTA an item (152 of them) with eight and sixteen rows; items over several CTAs; single-tile steps
shapes = pytest.mark.parametrize("B,Hkv,G", [(19, 8, 4), (19, 8, 16), (5, 3, 8), (1, 1, 4)])


@both
@shapes
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("peak", [None, 290, 1500])
def test_a_large_value_among_keys_of_no_weight(bsa, q8, B, Hkv, G, D, peak):  # noqa: F811
    """The first 144 slots 2^-70 in weight, one value row there 2^40 times the others."""
    score = [0.0 if s < 144 else 70.0 for s in range(N)]
    if peak is not None:
        score[peak] += 14
    size = [0.0] * N
    size[5] = 40.0
    c = steep_cache(D, Hkv, B, q8, score, size, B + G)
    check(bsa, c, queries(B, Hkv * G, D, 1.0, D), q8)


@both
@shapes
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rise,fall", [(100, 80), (100, 20), (100, 99), (20, 100)])
def test_growing_maxima_and_falling_values(bsa, q8, B, Hkv, G, D, rise, fall):  # noqa: F811
    """Scores rise by 2^rise from the first slot to the last while values fall by 2^fall; the heads'
    maxima grow at paces of their own, so that some follow in steps that others call for."""
    score = [rise * s / N for s in range(N)]
    size = [-fall * s / N for s in range(N)]
    c = steep_cache(D, Hkv, B, q8, score, size, rise + fall)
    first = torch.tensor([1.0, 0.5, 0.25, 0.75] * (Hkv * G // 4))
    check(bsa, c, queries(B, Hkv * G, D, first, D), q8)


@both
def test_the_ends_of_the_scales(bsa, q8):  # noqa: F811
    """Values from 2^86 down to 2^-114 under scores that rise as fast: every power of two in between is
    the largest product met at some slot."""
    score = [118.0 * s / N for s in range(N)]
    size = [86 - 200.0 * s / N for s in range(N)]
    c = steep_cache(128, 8, 19, q8, score, size, 1)
    check(bsa, c, queries(19, 32, 128, 1.0, 2), q8)
    # scores first, then values
    half = N // 2
    score = [-118.0 if s < half else 0.0 for s in range(N)]
    size = [86.0 if s < half else -20.0 for s in range(N)]
    c = steep_cache(128, 8, 19, q8, score, size, 2)
    check(bsa, c, queries(19, 32, 128, 1.0, 3), q8)


@both
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rise,fall", [(100, 80), (100, 20), (20, 100)])
def test_chunks_of_them(bsa, q8, D, rise, fall):  # noqa: F811
    """The same under chunks, whose weights are rounded to bf16."""
    n, B, Hkv, G = 40, 3, 2, 4
    score = [rise * s / N for s in range(N)]
    size = [-fall * s / N for s in range(N)]
    size[5] += 20
    c = steep_cache(D, Hkv, B, q8, score, size, rise)
    q = queries(B * n, Hkv * G, D, torch.tensor([1.0, 0.5, 0.25, 0.75] * (Hkv * G // 4)), D)
    k, v, table, sc = c.device()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ctx, ptr = [N - n] * B, [n * b for b in range(B + 1)]
    o, lse = bsa.chunk_attention(q.cuda(), k, v, table, i32(ctx), q_ptr=i32(ptr), **sc)
    assert bsa.device_error() == 0
    check_attention(o, lse, attention(c, q, ptr, ctx, 0, 0, D ** -0.5), D, 2.0 ** -8)
