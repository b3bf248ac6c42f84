"""tree_attention against softmax attention in 64 bits (torch, on the CPU).

Tolerances, derived before the first run, for O = sum p v / sum p with
A = sum p |v| / sum p:
  scores: fp32 sums of D products, each addition off by 2^-24 of a partial sum
    that is at most M = max over keys of scale * sum_d |q_d k_d|: D M 2^-24;
    the exponent's product, subtraction and 2^x: |x| 2^-23 + 2^-22, |x| <= 2 M
    -> relative error of a weight  e = (D + 4 * 2) M 2^-24 + 2^-21
  p is rounded to bf16 once: 2^-8; fp32 accumulation: steps * 2^-24, inside 2^-16
  O: A (2^-8 + 2 e + 2^-16) + |O| 2^-8 (its own rounding)
  LSE: e + 2^-21 (|LSE| + 1)
"""

import numpy as np
import pytest
import torch

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
    """Random pools whose unused slots and pages hold NaN, and the 64-bit answer."""

    def __init__(self, B, T, Hq, Hkv, D, page, ctx, dl=None, mask="tree", lists=None, seed=0, scale=None,
                 q_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.T, self.Hq, self.Hkv, self.D, self.page = B, T, Hq, Hkv, D, page
        self.ctx = [ctx] * B if isinstance(ctx, int) else list(ctx)
        self.dl = None if dl is None else list(dl)
        n = [c + (T if dl is None else dl[b]) for b, c in enumerate(self.ctx)]
        held = [-(-x // page) for x in n]
        P = max(1, max(held)) + 1
        n_pages = sum(held) + 3
        order = torch.randperm(n_pages, generator=g).int()
        self.table = torch.full((B, P), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            self.table[b, :held[b]] = order[at:at + held[b]]
            at += held[b]
        self.kc = torch.full((n_pages, Hkv, page, D), float("nan"), dtype=torch.bfloat16)
        self.vc = self.kc.clone()
        for b in range(B):
            for j in range(held[b]):
                r = min(page, n[b] - j * page)
                pg = int(self.table[b, j])
                self.kc[pg, :, :r] = torch.randn(Hkv, r, D, generator=g).bfloat16()
                self.vc[pg, :, :r] = torch.randn(Hkv, r, D, generator=g).bfloat16()
        self.q = (torch.randn(B, T, Hq, D, generator=g) * q_scale).bfloat16()
        self.mask = None
        if mask == "tree":
            self.mask = torch.zeros(B, T, dtype=torch.int64)
            for b in range(B):
                bits = []
                for u in range(T):
                    w = (bits[int(torch.randint(0, u, (1,), generator=g))] if u else 0) | 1 << u
                    bits.append(w)
                    self.mask[b, u] = w - (1 << 64) if w >> 63 else w
        elif mask == "none":
            self.mask = torch.zeros(B, T, dtype=torch.int64)
        elif mask == "all":
            self.mask = torch.full((B, T), -1, dtype=torch.int64)
        self.rp = self.ci = None
        if lists is not None:
            rp, ci = [0], []
            for b in range(B):
                for h in range(Hkv):
                    row = lists(b, h, held[b], g)
                    ci += row
                    rp.append(len(ci))
            self.rp, self.ci = torch.tensor(rp, dtype=torch.int32), torch.tensor(ci, dtype=torch.int32)
        self.scale = D ** -0.5 if scale is None else scale

    def run(self, bsa, stream=None, **kw):
        c = lambda t: None if t is None else t.cuda()
        dl = None if self.dl is None else torch.tensor(self.dl, dtype=torch.int32).cuda()
        self.dev = (self.q.cuda(), self.kc.cuda(), self.vc.cuda(), self.table.cuda(),
                    torch.tensor(self.ctx, dtype=torch.int32).cuda(), dl, c(self.mask), c(self.rp), c(self.ci))
        return bsa.tree_attention(*self.dev, scale=self.scale, stream=stream, **kw)

    def check(self, o, lse, only=None):
        B, T, Hq, Hkv, D, page = self.B, self.T, self.Hq, self.Hkv, self.D, self.page
        G = Hq // Hkv
        o, lse = o.detach().cpu().double(), lse.detach().cpu().double()
        worst = 0.0
        for b in range(B):
            n = T if self.dl is None else self.dl[b]
            end = self.ctx[b] + n
            for h in range(Hkv):
                js = list(range(-(-end // page)))
                if self.rp is not None:
                    r = b * Hkv + h
                    js = [int(x) for x in self.ci[self.rp[r]:self.rp[r + 1]]]
                    js = [j for j in js if 0 <= j and j * page < end]
                slots = torch.tensor([j * page + i for j in js for i in range(page) if j * page + i < end],
                                     dtype=torch.long)
                pg = self.table[b, slots // page].long()
                K = self.kc[pg, h, slots % page].double()
                V = self.vc[pg, h, slots % page].double()
                for t in range(n):
                    if self.mask is None:
                        bits = (1 << (t + 1)) - 1
                    else:
                        bits = int(self.mask[b, t]) & (2 ** 64 - 1)
                    see = torch.tensor([s < self.ctx[b] or bits >> (s - self.ctx[b]) & 1 for s in slots.tolist()],
                                       dtype=torch.bool)
                    q = self.q[b, t, h * G:(h + 1) * G].double()
                    go, gl = o[b, t, h * G:(h + 1) * G], lse[b, t, h * G:(h + 1) * G]
                    if not see.any():
                        assert (go == 0).all() and torch.isneginf(gl).all()
                        continue
                    S = q @ K[see].T * self.scale
                    L = torch.logsumexp(S, -1)
                    w = torch.exp(S - L[:, None])
                    O, A = w @ V[see], w @ V[see].abs()
                    M = (q.abs() @ K[see].abs().T * self.scale).amax(-1)
                    e = (D + 8) * M * 2.0 ** -24 + 2.0 ** -21
                    tol = A * (2.0 ** -8 + 2 * e[:, None] + 2.0 ** -16) + O.abs() * 2.0 ** -8
                    assert torch.isfinite(go).all(), (b, h, t)
                    r = ((go - O).abs() / tol).max().item()
                    d = ((gl - L).abs() / (e + 2.0 ** -21 * (L.abs() + 1))).max().item()
                    worst = max(worst, r, d)
                    assert r <= 1 and d <= 1, "sequence %d head %d draft %d: O %.3g LSE %.3g of the tolerance" % (
                        b, h, t, r, d)
        return worst


def listed(frac):
    def rows(b, h, held, g):
        n = max(0, min(held, int(held * frac) + h % 2))
        return torch.randperm(held, generator=g)[:n].tolist()
    return rows


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [64, 128])
@pytest.mark.parametrize("ctx", [0, 1, 63, 64, 127, 128, 200, 1000])
def test_decode(bsa, D, page, ctx):
    c = Case(2, 1, 8, 2, D, page, [ctx, max(0, ctx - 1)], mask=None, seed=ctx)
    c.check(*c.run(bsa))
    assert bsa.device_error() == 0


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (1, 3, 1), (1, 16, 16), (2, 5, 1), (3, 4, 2), (5, 16, 2), (7, 14, 2),
                                      (8, 128, 1), (13, 10, 1), (16, 8, 1), (33, 5, 1), (64, 4, 2), (64, 16, 2),
                                      (1, 128, 1), (2, 128, 1)])
@pytest.mark.parametrize("page", [64, 128])
def test_trees(bsa, T, Hq, Hkv, page):
    c = Case(2, T, Hq, Hkv, 128 if T % 2 else 64, page, [150, 61], seed=T + Hq)
    c.check(*c.run(bsa))
    assert bsa.device_error() == 0


@pytest.mark.parametrize("mask", [None, "none", "all", "tree"])
def test_masks(bsa, mask):
    """A chain, no draft seen (an empty row where there is no context either), all, a tree."""
    c = Case(3, 9, 4, 2, 64, 64, [0, 60, 128], mask=mask)
    c.check(*c.run(bsa))


def test_ragged_drafts_leave_the_rest_alone(bsa):
    c = Case(5, 8, 8, 2, 128, 128, [0, 300, 127, 5, 640], dl=[8, 0, 3, 1, 7])
    o = torch.full((5, 8, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, 8, 8), 5.0, device="cuda")
    got = c.run(bsa, out=o, lse=lse)
    assert got[0] is o and got[1] is lse
    c.check(o, lse)
    for b, n in enumerate(c.dl):
        assert (o[b, n:] == 3).all() and (lse[b, n:] == 5).all()


@pytest.mark.parametrize("B", [1, 2, 40, 200])
@pytest.mark.parametrize("page", [64, 128])
def test_ragged_batches(bsa, B, page):
    """Ranges that cut items, hold several, end inside pages."""
    r = np.random.default_rng(B)
    ctx = [int(x) for x in r.integers(0, 5000 if B < 10 else 700, B)]
    c = Case(B, 2, 4, 2, 128 if page == 64 else 64, page, ctx, dl=[int(x) for x in r.integers(0, 3, B)], seed=B)
    c.check(*c.run(bsa))
    assert bsa.device_error() == 0


def test_one_long_row_over_every_sm(bsa):
    c = Case(1, 1, 1, 1, 128, 128, 50000, mask=None)
    c.check(*c.run(bsa))
    c = Case(1, 4, 8, 1, 64, 64, 20011)
    c.check(*c.run(bsa))


@pytest.mark.parametrize("frac", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("page", [64, 128])
def test_block_lists(bsa, frac, page):
    """Lists in any order, some rows without an entry, unlisted pages NaN for the row's head."""
    c = Case(4, 3, 8, 4, 64, page, [900, 0, 333, 1500], lists=listed(frac), seed=int(frac * 10))
    for b in range(c.B):
        for h in range(c.Hkv):
            r = b * c.Hkv + h
            on = set(c.ci[c.rp[r]:c.rp[r + 1]].tolist())
            for j in range(c.table.shape[1]):
                if j not in on and c.table[b, j] >= 0:
                    c.kc[c.table[b, j], h] = float("nan")
                    c.vc[c.table[b, j], h] = float("inf")
    c.check(*c.run(bsa))
    assert bsa.device_error() == 0


def test_bad_entries_are_skipped_and_reported(bsa):
    c = Case(2, 1, 2, 2, 64, 64, [400, 400], mask=None, lists=lambda b, h, held, g: list(range(held)))
    P = c.table.shape[1]
    ci = c.ci.clone()
    c.ci[1], c.ci[9] = -3, P + 7                     # outside the table
    o, lse = c.run(bsa)
    assert bsa.device_error() == 2
    keep = c.ci.clone()
    keep[1], keep[9] = -3, 10 ** 6                   # what the reference drops
    c.ci = keep
    c.check(o, lse)
    # entries past the sequence's end are no error and add nothing
    c.ci = ci.clone()
    c.ci[2] = P - 1
    o, lse = c.run(bsa)
    assert bsa.device_error() == 0
    c.check(o, lse)
    # a decreasing row_ptr: an empty row
    c.ci = ci
    c.rp = c.rp.clone()
    c.rp[2] = 3
    o, lse = c.run(bsa)
    assert bsa.device_error() == 4
    assert (o[0, 0, 1] == 0).all() and torch.isneginf(lse[0, 0, 1])


def test_missing_pages_are_reported(bsa):
    c = Case(1, 1, 1, 1, 64, 64, [300], mask=None)
    full = c.table.clone()
    c.table[0, 2] = c.kc.shape[0]                    # past the pool
    o, lse = c.run(bsa)
    assert bsa.device_error() == 32
    c.rp, c.ci = torch.tensor([0, 4], dtype=torch.int32), torch.tensor([0, 1, 3, 4], dtype=torch.int32)
    c.table = full
    c.check(o, lse)                                  # as if that page were not listed
    # a context longer than the table
    c.rp = c.ci = None
    c.ctx = [c.table.shape[1] * 64 + 100]
    c.run(bsa)
    assert bsa.device_error() == 32


def test_extreme_scores(bsa):
    """One key far above the rest, scores of hundreds, and the reference of the
    running maximum rising over many steps."""
    c = Case(1, 2, 2, 1, 64, 128, 1300, q_scale=30.0)
    c.check(*c.run(bsa))
    c = Case(1, 1, 2, 1, 64, 64, 900, mask=None)
    for j in range(15):
        pg = int(c.table[0, j])
        c.kc[pg, 0] = (c.kc[pg, 0].float() * 0.05 + (j + 1) * 0.8 * torch.sign(c.q[0, 0, 0].float())).bfloat16()
    c.kc[int(c.table[0, 14]), :, 5:] = float("nan")
    c.vc[int(c.table[0, 14]), :, 5:] = float("nan")
    c.check(*c.run(bsa))


def test_many_units(bsa):
    """More units than one launch takes."""
    c = Case(2100, 1, 1, 1, 64, 64, [i % 70 for i in range(2100)], mask=None)
    c.check(*c.run(bsa))
    c = Case(700, 1, 4, 4, 64, 64, [i % 90 for i in range(700)], mask=None, lists=listed(1.0))
    c.check(*c.run(bsa))


def test_streams_graphs_and_overlap(bsa):
    """Two calls at once on two streams, a captured call replayed on new
    contents, and the same bits every time."""
    a, b = Case(3, 4, 8, 2, 128, 128, [3000, 100, 1777], seed=1), Case(6, 1, 8, 4, 128, 128, 2000, mask=None, seed=2)
    ra, rb = a.run(bsa), b.run(bsa)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(5):
        outs.append((bsa.tree_attention(*a.dev, scale=a.scale, stream=s1),
                     bsa.tree_attention(*b.dev, scale=b.scale, stream=s2)))
    torch.cuda.synchronize()
    for x, y in outs:
        assert torch.equal(x[0], ra[0]) and torch.equal(x[1], ra[1])
        assert torch.equal(y[0], rb[0]) and torch.equal(y[1], rb[1])
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        oa = bsa.tree_attention(*a.dev, scale=a.scale)
    with torch.cuda.graph(g2):
        ob = bsa.tree_attention(*b.dev, scale=b.scale)
    a.dev[4][1] = 0                                  # a shorter context, on the device
    a.ctx[1] = 0
    with torch.cuda.stream(s1):
        g1.replay()
    with torch.cuda.stream(s2):
        g2.replay()
    torch.cuda.synchronize()
    ref = bsa.tree_attention(*a.dev, scale=a.scale)
    assert torch.equal(oa[0], ref[0]) and torch.equal(oa[1], ref[1]) and torch.equal(ob[0], rb[0])
    assert bsa.device_error() == 0


def test_no_wait_runs_out(bsa):
    """Whole calls stay far below the 2 s that a pipeline wait may last (an end
    of the pipeline that waits in vain would still give the right numbers)."""
    import time
    c = Case(8, 1, 8, 2, 128, 128, [1500 + 100 * i for i in range(8)], mask=None)
    c.run(bsa)
    torch.cuda.synchronize()
    t = time.monotonic()
    bsa.tree_attention(*c.dev, scale=c.scale)
    torch.cuda.synchronize()
    assert time.monotonic() - t < 1.0 and bsa.device_error() == 0


def test_a_row_of_nan_stays_alone(bsa):
    """A query row that is no number gives NaN (O and LSE) and leaves the others their bits;
    contexts long enough to be split over SMs, and short ones."""
    c = Case(2, 3, 8, 2, 128, 128, [5000, 40])
    o, lse = c.run(bsa)
    good = o.clone(), lse.clone()
    c.q[0, 1, 2] = float("nan")
    c.q[1, 2, 7, 5] = float("inf")
    o, lse = c.run(bsa)
    assert o[0, 1, 2].isnan().all() and lse[0, 1, 2].isnan()
    assert o[1, 2, 7].isnan().all() and lse[1, 2, 7].isnan()
    keep = torch.ones(2, 3, 8, dtype=torch.bool, device="cuda")
    keep[0, 1, 2] = keep[1, 2, 7] = False
    assert torch.equal(o[keep], good[0][keep]) and torch.equal(lse[keep], good[1][keep])


@pytest.mark.parametrize("ctx,dl", [(-5, 2), (3, -1), (3, 99)])
def test_lengths_out_of_range_are_clamped(bsa, ctx, dl):
    """A negative context is empty, drafts are taken as 0 .. T."""
    c = Case(1, 4, 2, 1, 64, 64, [10], dl=[4])
    c.ctx, c.dl = [ctx], [dl]
    o = torch.full((1, 4, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, 4, 2), 5.0, device="cuda")
    c.run(bsa, out=o, lse=lse)
    c.ctx, c.dl = [max(ctx, 0)], [min(max(dl, 0), 4)]
    c.check(o, lse)
    n = c.dl[0]
    assert (o[0, n:] == 3).all() and (lse[0, n:] == 5).all() and bsa.device_error() == 0


@pytest.mark.parametrize("D,page,T,Hq,Hkv", [(128, 64, 64, 8, 1), (64, 128, 40, 20, 4), (128, 128, 7, 96, 3),
                                             (64, 64, 33, 4, 2)])
def test_block_lists_of_several_row_tiles(bsa, D, page, T, Hq, Hkv):
    c = Case(3, T, Hq, Hkv, D, page, [700, 3, 1234], dl=[T, T - 1, 2], lists=listed(0.6), seed=T)
    o, lse = c.run(bsa)
    c.check(o, lse)
    assert bsa.device_error() == 0


def test_far_pages(bsa):
    """Rows whose offset in the pool passes 2^31 bytes and 2^30 elements: a pool of
    5 GB of which a few pages are used."""
    c = Case(2, 2, 8, 4, 128, 128, [400, 130], seed=4)
    want = c.run(bsa)
    n = 5 * 2 ** 30 // (4 * 128 * 128 * 2)
    big = [torch.empty(n, 4, 128, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    used = c.kc.shape[0]
    place = torch.arange(used) * (n // used) + (n // used - 1)
    for pool, small in zip(big, (c.kc, c.vc)):
        pool[place.cuda()] = small.cuda()
    table = c.dev[3].clone()
    table[table >= 0] = place.int().cuda()[table[table >= 0].long()]
    got = bsa.tree_attention(c.dev[0], big[0], big[1], table, *c.dev[4:], scale=c.scale)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and bsa.device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hq,Hkv", [
    (1, 1, 1), (1, 31, 1), (4, 16, 2), (3, 11, 1), (8, 16, 2), (5, 13, 1), (1, 96, 1), (1, 97, 1), (2, 64, 1),
    (3, 43, 1), (64, 16, 2), (64, 128, 1)])
def test_row_counts(bsa, D, T, Hq, Hkv):
    """Query rows of a key head on both sides of every change of layout (32, 64, 96
    and 128 rows), and up to 64 tiles of 128."""
    page = 64 if T % 2 else 128
    c = Case(4, T, Hq, Hkv, D, page, [0, 127, 129, 1000], dl=[T, T, max(T - 1, 1), 1], seed=Hq + T)
    got = []
    for _ in range(2):  # rows behind the drafts stay as they were: zeros
        o, lse = torch.zeros(4, T, Hq, D, dtype=torch.bfloat16).cuda(), torch.zeros(4, T, Hq).cuda()
        got.append(c.run(bsa, out=o, lse=lse))
    c.check(*got[0])
    assert all(torch.equal(x, y) for x, y in zip(*got)) and bsa.device_error() == 0


def test_long_items_outlast_the_wait_limit(bsa):
    """Contexts whose item keeps a CTA busy for longer than a pipeline wait may last
    (all logical pages are a few physical ones)."""
    B, P, n_pages = 4, 4000, 64
    g = torch.Generator().manual_seed(3)
    q = torch.randn(B, 2, 32, 128, generator=g).bfloat16().cuda()
    k, v = (torch.randn(n_pages, 8, 128, 128, generator=g).bfloat16().cuda() for _ in range(2))
    table = torch.randint(0, n_pages, (B, P), generator=g).int().cuda()
    ctx = torch.full((B,), P * 128 - 70, dtype=torch.int32).cuda()
    want = bsa.tree_attention(q, k, v, table, ctx)
    torch.cuda.synchronize()
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    bsa.set_wait_limit(150_000)
    try:
        t0.record()
        got = bsa.tree_attention(q, k, v, table, ctx)
        t1.record()
        torch.cuda.synchronize()
    finally:
        bsa.set_wait_limit(0)
    assert bsa.device_error() == 0 and t0.elapsed_time(t1) > 0.3
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
