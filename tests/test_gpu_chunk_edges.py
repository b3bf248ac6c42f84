"""Chunk attention, reading back and 8-bit appending at their borders: the short
form's, pools behind 2^32 bytes, many groups of one sequence, calls after one
another without a stop, captured steps.

Tolerances are test_gpu_chunk's; where a call is compared with itself (other pages,
another stream, a replay) the results are the same bits.
"""

import pytest
import torch

from paged_reference import E4M3, E8M0, Cache, attention, check_attention, quantise
from test_gpu_chunk import Case, both, bsa  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ the short form's border
@both
@pytest.mark.parametrize("G,new", [(16, [1]), (17, [1]), (8, [2]), (5, [3]), (5, [4]), (1, [16]), (1, [17]), (16, [1, 1]),
                                   (8, [2, 2]), (15, [1, 2]), (128, [1]), (128, [3, 0, 1])], ids=str)
def test_rows_at_the_border(bsa, q8, G, new):  # noqa: F811
    c = Case([70 * (i + 1) for i in range(len(new))], new, 2 * G, 2, 64, 64, q8, seed=G)
    c.short = [sum(new) * G <= 16] * len(new)  # with q_ptr
    c.check(*c.run(bsa))


@both
@pytest.mark.parametrize("G", [15, 16, 17])
def test_border_beside_chunks(bsa, q8, G):  # noqa: F811
    """A table that is wide enough for both kernels."""
    c = Case([500, 0, 64, 1000], [1, 40, 2, 1], 2 * G, 2, 64, 128, q8, table_extra=2000, seed=G)
    c.check(*c.run(bsa))


# ------------------------------------------------------------ one sequence of many groups
@both
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 5)])
def test_more_than_a_thousand_groups(bsa, q8, window, sinks):  # noqa: F811
    n, Hq, D = 2100, 70, 64  # a group is two tokens
    g = torch.Generator().manual_seed(7)
    cache = Cache([n], 1, D, 64, q8, 3)
    q = torch.randn(n, Hq, D, generator=g).bfloat16()
    k, v, table, sc = cache.device()
    o, lse = bsa.chunk_attention(q.cuda(), k, v, table, i32([0]), q_ptr=i32([0, n]), window=window, sinks=sinks, **sc)
    assert bsa.device_error() == 0
    for t in (0, 1000, 2047, 2080):
        m = min(20, n - t)
        ref = attention(cache, q[t:t + m], [0, m], [t], window, sinks, D ** -0.5)
        check_attention(o[t:t + m], lse[t:t + m], ref, D, 2.0 ** -8)


# ------------------------------------------------------------ pools behind 2^32 bytes
@both
def test_far_pages(bsa, q8):  # noqa: F811
    """The last pages of large pools give the same bits as those of small ones: append, attend, read."""
    Hkv, D, page, far = 8, 128, 64, 66000  # 2^32 codes and more
    c = Case([300, 100, 0], [1, 90, 40], 16, Hkv, D, page, q8)
    (q, k, v, table, ctx), more = c.args()
    n = k.shape[0]
    pools = [k, v] + [more[x] for x in ("k_scale", "v_scale") if x in more]
    big = [torch.empty(far, *x.shape[1:], dtype=x.dtype, device="cuda") for x in pools]
    for x, y in zip(big, pools):
        x.view(torch.uint8 if q8 else torch.bfloat16)[far - n:] = y.view(torch.uint8 if q8 else torch.bfloat16)
    table2 = torch.where(table >= 0, table + (far - n), table)
    sc, sc2 = (dict(zip(("k_scale", "v_scale"), p[2:])) for p in (pools, big))
    a = dict(q_ptr=more["q_ptr"])
    for x, y in zip(bsa.chunk_attention(q, k, v, table, ctx, **a, **sc), bsa.chunk_attention(q, *big[:2], table2, ctx, **a, **sc2)):
        assert torch.equal(x, y)
    one = q[:3].contiguous()
    for x, y in zip(bsa.chunk_attention(one, k, v, table, ctx, **sc), bsa.chunk_attention(one, *big[:2], table2, ctx, **sc2)):
        assert torch.equal(x, y)
    for x, y in zip(bsa.cache_read(k, v, table, i32([1, 0]), i32([190, 301]), 320, **sc),
                    bsa.cache_read(*big[:2], table2, i32([1, 0]), i32([190, 301]), 320, **sc2)):
        assert torch.equal(x, y)
    new = torch.randn(5, 32, D, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    seq, slot = i32([0, 1, 2, 0, 1]), i32([3, 64, 39, 300, 127])
    inv = bsa.rope_inv_freq(D)
    z = [bsa.cache_append(new[:, :16], new[:, 16:24], new[:, 24:], *p[:2], t, seq, slot, inv, **s)
         for p, t, s in ((pools, table, sc), (big, table2, sc2))]
    assert torch.equal(*z) and bsa.device_error() == 0
    for x, y in zip(big, pools):
        assert torch.equal(x.view(torch.uint8)[far - n:], y.view(torch.uint8))


# ------------------------------------------------------------ values of far magnitudes
def set_row(cache, b, slot, which, value):
    """Every head's K or V row of a slot to one value."""
    pg, at = int(cache.table[b, slot // cache.page]), slot % cache.page
    y = torch.full((cache.D,), value, dtype=torch.float64)
    pool = getattr(cache, which)
    if cache.q8:
        codes, e = quantise(y)
        pool[pg, :, at] = codes
        getattr(cache, which + "s")[pg, :, at] = e
    else:
        pool[pg, :, at] = y.bfloat16()


@both
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_values_of_far_magnitudes(bsa, q8, n, D):  # noqa: F811
    """Rows whose values are 2^50 times the others' and whose weight is 2^-78 (a window's hidden
    rows: 2^100 and none) drown nothing; nor do heads that see large values the others."""
    G, ctx, page = 4, 300, 64
    g = torch.Generator().manual_seed(n)
    for window in (0, 100):
        cache = Cache([ctx + n], 1, D, page, q8, 5)
        for slot in (7, 130, 290):
            set_row(cache, 0, slot, "k", -48.0 / D ** 0.5)
            set_row(cache, 0, slot, "v", 2.0 ** 50)
        if window:
            set_row(cache, 0, 195, "v", 2.0 ** 100)  # a page that is read, in front of every window
        q = torch.randn(n, G, D, generator=g).abs().bfloat16()
        q[:, 2] = -q[:, 2] / 4  # sees the large values
        k, v, table, sc = cache.device()
        ptr = None if n == 1 else i32([0, n])
        o, lse = bsa.chunk_attention(q.cuda(), k, v, table, i32([ctx]), q_ptr=ptr, window=window, **sc)
        assert bsa.device_error() == 0
        ref = attention(cache, q, [0, n], [ctx], window, 0, D ** -0.5)
        check_attention(o, lse, ref, D, 2.0 ** -8 if n > 1 else 2.0 ** -11 if q8 else 2.0 ** -16)


# ------------------------------------------------------------ one call after another
@both
def test_back_to_back(bsa, q8):  # noqa: F811
    """Short, mixed and long batches in turn, no stop between: each as it is alone."""
    cs = [Case([900, 20, 300], [1, 1, 1], 8, 2, 128, 64, q8), Case([0, 700], [333, 2], 8, 2, 128, 64, q8, window=100, sinks=3),
          Case([40] * 30, [1, 0, 17] * 10, 4, 4, 64, 128, q8), Case([1500], [64], 40, 2, 64, 64, q8),
          Case([2000, 100, 0, 64], [1, 200, 1, 1], 16, 4, 128, 128, q8, table_extra=600)]
    cs[0].short = [False] * 3  # with q_ptr
    args = [c.args() for c in cs]
    first = [bsa.chunk_attention(*a, **m) for a, m in args]
    for c, r in zip(cs, first):
        c.check(*r)
    last = None
    for _ in range(40):
        last = [bsa.chunk_attention(*a, **m) for a, m in args]
    torch.cuda.synchronize()
    assert bsa.device_error() == 0
    for x, y in zip(first, last):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


# ------------------------------------------------------------ captured steps
@both
def test_captured_decoding_step(bsa, q8):  # noqa: F811
    """Append and attend in one graph, replayed with lengths, tokens and pages that change between replays."""
    Hq, Hkv, D, page, B, P = 8, 2, 128, 64, 3, 6
    g = torch.Generator().manual_seed(11)
    dt = E4M3 if q8 else torch.bfloat16
    table = i32([[5 * b + j for j in range(5)] + [-1] for b in range(B)])
    inv, w = bsa.rope_inv_freq(D), torch.ones(D, device="cuda")
    seq = torch.arange(B, dtype=torch.int32, device="cuda")

    def fresh():
        kc, vc = (torch.zeros(5 * B, Hkv, page, D, dtype=dt, device="cuda") for _ in range(2))
        if not q8:
            return kc, vc, {}
        s = [torch.full((5 * B, Hkv, page), 127, dtype=torch.uint8, device="cuda").view(E8M0) for _ in range(2)]
        return kc, vc, dict(k_scale=s[0], v_scale=s[1])

    def step(x, ctx, kc, vc, sc, **kw):
        q = bsa.cache_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kc, vc, table, seq, ctx, inv, q_weight=w,
                             k_weight=w, **sc, **kw)
        return bsa.chunk_attention(q, kc, vc, table, ctx, window=200, sinks=2, **sc, **kw)

    xs = [torch.randn(B, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda() for _ in range(70)]
    a, b = fresh(), fresh()
    x, ctx = xs[0].clone(), i32([0, 100, 250])
    warm = fresh()
    step(x, ctx, *warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step(x, ctx, *a)
    side = torch.cuda.Stream()
    for i, new in enumerate(xs):
        x.copy_(new)
        ctx.copy_(i32([i, 100 + i, 250 + i]))
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        o2, l2 = step(new, ctx, *b, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and bsa.device_error() == 0


# ------------------------------------------------------------ given outputs
@both
def test_given_outputs_and_refused_ones(bsa, q8):  # noqa: F811
    c = Case([100, 3], [30, 1], 4, 2, 64, 64, q8)
    (q, k, v, table, ctx), more = c.args()
    o, l = torch.empty_like(q), torch.empty(31, 4, device="cuda")
    r = bsa.chunk_attention(q, k, v, table, ctx, out=o, lse=l, **more)
    assert r[0].data_ptr() == o.data_ptr() and r[1].data_ptr() == l.data_ptr()
    c.check(o, l)
    wide = torch.empty(31, 4, 128, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(out=wide[..., :64]), dict(out=o.float()), dict(out=o[:30]), dict(lse=l.T.contiguous().T), dict(lse=l.double()),
                dict(out=o.cpu())):
        with pytest.raises(ValueError):
            bsa.chunk_attention(q, k, v, table, ctx, **{**more, **bad})
    for bad in (wide[..., :64], q.float(), q[None], q.cpu()):
        with pytest.raises(ValueError):
            bsa.chunk_attention(bad, k, v, table, ctx, **more)
    for bad in (dict(window=-1), dict(sinks=-2), dict(scale=0.0), dict(scale=float("nan")), dict(q_ptr=None),
                dict(q_ptr=more["q_ptr"].long()), dict(q_ptr=more["q_ptr"][:2])):
        with pytest.raises((ValueError, RuntimeError)):
            bsa.chunk_attention(q, k, v, table, ctx, **{**more, **bad})
    sc = {x: more[x] for x in ("k_scale", "v_scale") if x in more}
    for bad in (dict(n=-1), dict(kv_repeat=0), dict(lens=i32([1])), dict(lens=i32([1, 2]).long()), dict(first=i32([1])),
                dict(out=(q,)), dict(seq_ids=i32([0, 1]).cpu())):
        a = {**dict(seq_ids=i32([0, 1]), lens=None, n=64), **sc, **bad}
        with pytest.raises((ValueError, RuntimeError, TypeError)):
            bsa.cache_read(k, v, table, **a)
    assert bsa.device_error() == 0
