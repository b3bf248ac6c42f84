"""chunk_attention against softmax attention in 64 bits (torch, on the CPU).

Tolerances, derived before the first run, for O = sum p v / sum p with
A = sum p |v| / sum p:
  scores: fp32 sums of D products, each addition off by 2^-24 of a partial sum
    that is at most M = max over keys of scale * sum_d |q_d k_d|: D M 2^-24;
    the exponent's product, subtraction and 2^x: |x| 2^-23 + 2^-22, |x| <= 2 M
    -> relative error of a weight  e = (D + 4 * 2) M 2^-24 + 2^-21
  p is rounded to bf16 once, 2^-8 (chunks, and the short sequences of a small batch
    that has chunks too); in short sequences of up to 16 rows a key head it is held in
    two bf16 parts, 2^-16, or, times the 8-bit row's scale, rounded to fp16 once,
    2^-11 (below fp16's normal numbers, 2^-20 of the largest such product: off by 2^-31
    of that, inside 2^-16); fp32 accumulation: steps * 2^-24, inside 2^-16
  O: A (p's + 2 e + 2^-16) + |O| 2^-8 (its own rounding)
  LSE: e + 2^-21 (|LSE| + 1)
8-bit rows are what they are (code * 2^e): the reference reads the same values.
"""

import math

import pytest
import torch

from paged_reference import Cache, attention, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_flashattention_bsa_gb300 import build
    build.build()
    import block_sparse_flashattention_bsa_gb300 as m
    m.device_error()
    return m


class Case:
    def __init__(self, ctx, new, Hq, Hkv, D, page, q8, window=0, sinks=0, seed=0, q_scale=1.0, spread=1.0, release=False,
                 table_extra=1):
        g = torch.Generator().manual_seed(seed + 1)
        self.ctx, self.new, self.window, self.sinks, self.D = list(ctx), list(new), window, sinks, D
        self.cache = Cache([c + n for c, n in zip(ctx, new)], Hkv, D, page, q8, seed, spread=spread,
                           table_extra=table_extra)
        self.q_ptr = [0]
        for n in new:
            self.q_ptr.append(self.q_ptr[-1] + n)
        self.q = (torch.randn(self.q_ptr[-1], Hq, D, generator=g) * q_scale).bfloat16()
        self.ref = attention(self.cache, self.q, self.q_ptr, self.ctx, window, sinks, D ** -0.5)
        if release:  # pages that no new token sees any more are given back
            for b, c in enumerate(ctx):
                for j in range(-(-c // page)):
                    if (j + 1) * page <= c - window + 1 and j * page >= sinks:
                        self.cache.table[b, j] = -1
        self.G = Hq // Hkv
        # whose rows the short form takes: all, or those of a batch of some size
        P = self.cache.table.shape[1] * page / 128
        alone = sum(new) * self.G <= 16 or (max(new) == 1 and self.G <= 16)
        self.short = [n * self.G <= 16 and (alone or len(ctx) * P * Hkv > 64 * 160) for n in new]

    def args(self, one=False):
        k, v, table, sc = self.cache.device()
        ctx = torch.tensor(self.ctx, dtype=torch.int32).cuda()
        ptr = None if one else torch.tensor(self.q_ptr, dtype=torch.int32).cuda()
        return (self.q.cuda(), k, v, table, ctx), dict(q_ptr=ptr, window=self.window, sinks=self.sinks, **sc)

    def run(self, bsa, one=False, **kw):
        a, more = self.args(one)
        o, lse = bsa.chunk_attention(*a, **more, **kw)
        torch.cuda.synchronize()
        assert bsa.device_error() == 0
        return o, lse

    def check(self, o, lse):
        """Short sequences and the others to their own tolerance."""
        for b, (r, n) in enumerate(zip(self.q_ptr, self.new)):
            if n:
                part = [x[r:r + n] for x in self.ref]
                p = 2.0 ** -8 if not self.short[b] else 2.0 ** -11 if self.cache.q8 else 2.0 ** -16
                check_attention(o[r:r + n], lse[r:r + n], part, self.D, p)


both = pytest.mark.parametrize("q8", [False, True], ids=["bf16", "q8"])
sizes = pytest.mark.parametrize("D,page", [(64, 64), (64, 128), (128, 64), (128, 128)])


# ------------------------------------------------------------ one token a sequence
@both
@sizes
@pytest.mark.parametrize("G", [1, 4, 5, 8])
def test_decoding(bsa, D, page, q8, G):
    ctx = [0, 1, 62, 63, 64, 127, 128, 129, 300, 1000, 2049]
    c = Case(ctx, [1] * len(ctx), 2 * G, 2, D, page, q8, seed=G)
    c.check(*c.run(bsa, one=True))
    c.short = [False] * len(ctx)
    c.check(*c.run(bsa))  # the same with q_ptr


@both
@pytest.mark.parametrize("D,G", [(64, 16), (128, 12), (128, 16)])
def test_decoding_sixteen_rows(bsa, D, q8, G):
    ctx = [5, 127, 700, 1500]
    c = Case(ctx, [1] * 4, G, 1, D, 64, q8, seed=G)
    c.check(*c.run(bsa, one=True))


@both
def test_few_tokens_short(bsa, q8):
    """Two to eight tokens of few heads: still the short form."""
    c = Case([0, 3, 120, 500, 129], [2, 8, 5, 3, 1], 4, 2, 128, 64, q8)
    c.check(*c.run(bsa))
    for n in (2, 5, 8):
        c = Case([140], [n], 2, 1, 128, 64, q8, seed=n)
        assert all(c.short)
        c.check(*c.run(bsa))


@both
def test_decoding_long_context(bsa, q8):
    """Over all SMs: every CTA has a part of the one item or two."""
    c = Case([40000], [1], 4, 1, 128, 128, q8)
    c.check(*c.run(bsa, one=True))


@both
def test_few_tokens_beside_chunks(bsa, q8):
    """Small batches; then a table wide enough for both forms: each row to its own tolerance."""
    new = [1, 2, 1, 70, 1, 4, 1, 1, 300, 1, 0, 1] * 2
    c = Case([3000 + 7 * b for b in range(24)], new, 8, 4, 128, 64, q8)
    c.check(*c.run(bsa))
    c = Case([1000 + 97 * b for b in range(24)], new, 8, 4, 128, 64, q8, table_extra=200)
    assert any(c.short) and not all(c.short)
    for _ in range(5):
        c.check(*c.run(bsa))


@both
def test_ends_of_sequences_in_flight(bsa, q8):
    """Many items a CTA, each with a last tile of rows that are not there (NaN), again and again."""
    for D, page in ((128, 64), (64, 128), (128, 128)):
        c = Case([3000 + 7 * b for b in range(16)], [70, 1, 2, 130] * 4, 8, 4, D, page, q8)
        for _ in range(5):
            o, lse = c.run(bsa)
        c.check(o, lse)


@both
def test_many_sequences(bsa, q8):
    """More than one launch's worth, most of them of one step."""
    g = torch.Generator().manual_seed(3)
    ctx = torch.randint(0, 140, (1100,), generator=g).tolist()
    c = Case(ctx, [1] * 1100, 2, 1, 64, 64, q8)
    c.check(*c.run(bsa, one=True))


# ------------------------------------------------------------ chunks
@both
@sizes
@pytest.mark.parametrize("G", [1, 4, 5, 8])
def test_chunks(bsa, D, page, q8, G):
    c = Case([0, 17, 200, 128], [100, 33, 129, 64], 2 * G, 2, D, page, q8, seed=G)
    c.check(*c.run(bsa))


@both
@pytest.mark.parametrize("n", [17, 127, 128, 129, 255, 256, 257, 700])
def test_chunk_lengths(bsa, q8, n):
    c = Case([77], [n], 1, 1, 128, 64, q8, seed=n)
    c.check(*c.run(bsa))


@both
@pytest.mark.parametrize("G", [17, 33, 64, 65, 100, 128])
def test_many_heads(bsa, q8, G):
    """Single tokens and chunks of groups that the short form does not take."""
    c = Case([0, 130, 500], [1, 1, 5], G, 1, 128, 64, q8, seed=G)
    c.check(*c.run(bsa))
    d = Case([0, 130], [1, 1], G, 1, 64, 128, q8, seed=G)
    d.check(*d.run(bsa, one=True))


@both
def test_mixed_batch(bsa, q8):
    """Single tokens, chunks, and sequences that bring nothing."""
    ctx = [900, 0, 33, 250, 0, 1300, 64, 5]
    new = [1, 140, 0, 1, 1, 60, 0, 3]
    c = Case(ctx, new, 8, 2, 128, 64, q8)
    c.check(*c.run(bsa))


@both
def test_long_prefix(bsa, q8):
    """Few rows behind a long prefix: items are split over the SMs."""
    c = Case([20000], [40], 8, 2, 128, 128, q8)
    c.check(*c.run(bsa))


@both
def test_large_scores(bsa, q8):
    """The reference has to follow maxima that grow by more than 2^8 again and again."""
    c = Case([600, 40], [150, 1], 4, 1, 64, 64, q8, q_scale=20.0, spread=1.5)
    c.check(*c.run(bsa))


# ------------------------------------------------------------ window and sinks
@both
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (50, 4), (128, 0), (129, 130), (300, 64), (5000, 4), (64, 5000)])
def test_window(bsa, q8, window, sinks):
    c = Case([0, 40, 700, 130], [150, 1, 200, 90], 4, 1, 128, 64, q8, window, sinks, seed=window)
    c.check(*c.run(bsa))


@both
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 4), (129, 130)])
def test_window_decoding(bsa, q8, window, sinks):
    c = Case([0, 40, 700, 1300, 127], [1] * 5, 8, 2, 64, 128, q8, window, sinks, seed=window)
    c.check(*c.run(bsa, one=True))


@both
@pytest.mark.parametrize("new", [1, 120])
def test_window_over_released_pages(bsa, q8, new):
    c = Case([900, 2000], [new, 1], 4, 2, 64, 64, q8, 200, 70, release=True)
    assert (c.cache.table[0, :10] < 0).any()
    c.check(*c.run(bsa))


# ------------------------------------------------------------ edges
@both
def test_rows_of_no_sequence_are_left(bsa, q8):
    c = Case([100, 30], [1, 50], 4, 2, 128, 64, q8)
    (q, k, v, table, ctx), more = c.args()
    pad = 7
    q2 = torch.cat([q[:pad], q, q[:9]])
    ptr = more.pop("q_ptr") + pad
    o = torch.full_like(q2, 3.0)
    l = torch.full(q2.shape[:2], 5.0, device="cuda")
    bsa.chunk_attention(q2, k, v, table, ctx, q_ptr=ptr, out=o, lse=l, **more)
    assert bsa.device_error() == 0
    n = q.shape[0]
    assert (o[:pad] == 3).all() and (o[pad + n:] == 3).all() and (l[:pad] == 5).all() and (l[pad + n:] == 5).all()
    c.check(o[pad:pad + n], l[pad:pad + n])


@both
def test_missing_pages_are_reported(bsa, q8):
    """A page that should be there: its slots are not seen, the error word says so."""
    c = Case([300, 200], [1, 70], 4, 1, 64, 64, q8)
    (q, k, v, table, ctx), more = c.args()
    table[0, 1], table[1, 0] = -1, 10 ** 6
    o, lse = bsa.chunk_attention(q, k, v, table, ctx, **more)
    assert bsa.device_error() == 32
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    d = Case([300, 200], [1, 70], 4, 1, 64, 64, q8)
    for b, j, pos in ((0, 1, 300), (1, 0, 200)):
        slots = torch.tensor([s for s in range(pos + 1) if s // 64 != j])
        K, V = d.cache.rows(b, 0, slots)
        S = d.q[c.q_ptr[b], 0].double() @ K.T / 8
        assert abs(torch.logsumexp(S, -1).item() - lse[c.q_ptr[b], 0].item()) < 1e-4
    table[:] = -1  # nothing is there: zeros
    o, lse = bsa.chunk_attention(q, k, v, table, ctx, **more)
    assert bsa.device_error() == 32
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_positions_behind_the_table_are_reported(bsa):
    c = Case([300, 10], [1, 40], 4, 1, 64, 64, False)
    (q, k, v, table, ctx), more = c.args()
    ctx[0] = 64 * table.shape[1] + 5
    o, lse = bsa.chunk_attention(q, k, v, table, ctx, **more)
    assert bsa.device_error() & 32
    ctx[0] = 2 ** 31 - 1
    bsa.chunk_attention(q, k, v, table, ctx, **more)
    assert bsa.device_error() & 32
    check_attention(o[1:], lse[1:], [x[1:] for x in c.ref], 64, 2.0 ** -8)


@pytest.mark.parametrize("ptr", [[0, 50, 20], [-1, 10, 20], [0, 10, 200], [5, 2, 2 ** 31 - 1]])
def test_bad_row_pointers_are_reported(bsa, ptr):
    c = Case([100, 30], [40, 10], 4, 1, 64, 64, False)
    (q, k, v, table, ctx), more = c.args()
    more["q_ptr"] = torch.tensor(ptr, dtype=torch.int32).cuda()
    o = torch.full_like(q, 3.0)
    l = torch.full(q.shape[:2], 5.0, device="cuda")
    bsa.chunk_attention(q, k, v, table, ctx, out=o, lse=l, **more)
    assert bsa.device_error() & 4
    left = torch.ones(50, dtype=torch.bool)
    for lo, hi in zip(ptr, ptr[1:]):
        if 0 <= lo <= hi <= 50:
            left[lo:hi] = False
    assert left.any() or ptr[1] == 50
    assert (o.cpu()[left] == 3).all() and (l.cpu()[left] == 5).all() and (l.cpu()[~left] != 5).all()


def test_empty(bsa):
    kc = torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    o, l = bsa.chunk_attention(torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda"), kc, kc,
                               torch.zeros(0, 3, dtype=torch.int32, device="cuda"), i32())
    assert o.shape == (0, 4, 64) and l.shape == (0, 4)
    o, l = bsa.chunk_attention(torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda"), kc, kc,
                               torch.zeros(2, 3, dtype=torch.int32, device="cuda"), i32(5, 6), q_ptr=i32(0, 0, 0))
    assert o.shape == (0, 4, 64) and bsa.device_error() == 0


# ------------------------------------------------------------ how it is called
def case_of_both(q8, seed=0):
    return Case([300, 0, 129, 1000], [1, 150, 1, 40], 8, 2, 128, 64, q8, seed=seed)


@both
def test_same_answer_every_time(bsa, q8):
    c = case_of_both(q8)
    o, l = c.run(bsa)
    for _ in range(3):
        o2, l2 = c.run(bsa)
        assert torch.equal(o, o2) and torch.equal(l, l2)


@both
def test_streams_and_graphs(bsa, q8):
    """Two streams at once, and two captured calls whose workspaces are their own."""
    cs = [case_of_both(q8, seed) for seed in (1, 2)]
    args = [c.args() for c in cs]
    s = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        outs = [bsa.chunk_attention(*a, **m, stream=st) for (a, m), st in zip(args, s)]
    torch.cuda.synchronize()
    for c, r in zip(cs, outs):
        c.check(*r)
    graphs, outs = [], []
    for (a, m) in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(bsa.chunk_attention(*a, **m))
        graphs.append(g)
    for o, l in outs:
        o.zero_()
        l.zero_()
    torch.cuda.synchronize()
    for g, st in zip(graphs, s):
        with torch.cuda.stream(st):
            g.replay()
    torch.cuda.synchronize()
    for c, r in zip(cs, outs):
        c.check(*r)
    assert bsa.device_error() == 0


def test_against_tree_attention(bsa):
    """Chains of drafts are chunks: the two calls agree within their roundings."""
    c = Case([500, 90], [8, 8], 8, 2, 128, 64, False)
    (q, k, v, table, ctx), more = c.args()
    o, l = bsa.chunk_attention(q, k, v, table, ctx, **more)
    o2, l2 = bsa.tree_attention(q.reshape(2, 8, 8, 128), k, v, table, ctx)
    check_attention(o2.reshape(o.shape), l2.reshape(l.shape), c.ref, 128, 2.0 ** -8)
    c.check(o, l)
