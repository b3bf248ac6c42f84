"""The pages of the cache: resize, fork, compact, accept against a plain Python
model of the table, the counts and the rows.  Everything is exact."""

import random

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


class Model:
    """The rules of include/bsa.h, one request after the other."""

    def __init__(self, S, P, pages, layers=2, Hkv=3, page=64, D=64, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.S, self.P, self.pages, self.page = S, P, pages, page
        self.table = [[-1] * P for _ in range(S)]
        self.ref = [0] * pages
        self.k, self.v = (torch.randn(layers, pages, Hkv, page, D, generator=g).bfloat16() for _ in range(2))
        if layers == 1:
            self.k, self.v = self.k[0], self.v[0]
        self.dt = torch.tensor(self.table, dtype=torch.int32).cuda()
        self.dr = torch.tensor(self.ref, dtype=torch.int32).cuda()
        self.dk, self.dv = self.k.cuda(), self.v.cuda()

    def held(self, s):
        row = self.table[s]
        return row.index(-1) if -1 in row else self.P

    def copy(self, src, dst, rows):
        for t in (self.k, self.v):
            t = t if t.dim() == 5 else t[None]
            t[:, dst, :, :rows] = t[:, src, :, :rows]

    def serve(self, reqs, plan):
        """plan(request, ref at the start, table at the start) -> None or (need, apply(fresh))."""
        ref0, table0 = list(self.ref), [list(r) for r in self.table]
        free = [p for p in range(self.pages) if ref0[p] == 0]
        seen, used, granted, todo = set(), 0, [], []
        for r in reqs:
            got = plan(r, ref0, table0) if 0 <= r[0] < self.S and r[0] not in seen else None
            if 0 <= r[0] < self.S:
                seen.add(r[0])
            ok = False
            if got is not None:
                need, apply = got
                if need == 0 or used + need <= len(free):
                    todo.append((apply, free[used:used + need]))
                    ok = True
                used += need
            granted.append(int(ok))
        for apply, fresh in todo:
            apply(fresh)
        return granted

    def resize(self, reqs):
        pg = self.page

        def plan(r, ref0, table0):
            s, keep, cap = r
            if not (0 <= keep <= cap <= self.P * pg):
                return None
            row, held = table0[s], (table0[s].index(-1) if -1 in table0[s] else self.P)
            full, part, want = keep // pg, keep % pg, -(-cap // pg)
            first = full + (part > 0)
            if first > held or any(not 0 <= row[j] < self.pages or ref0[row[j]] <= 0 for j in range(held)):
                return None
            cow = part and ref0[row[full]] > 1
            take = [j for j in range(first, want) if j >= held or ref0[row[j]] != 1]

            def apply(fresh):
                fresh = list(fresh)
                if cow:
                    p = fresh.pop(0)
                    self.copy(row[full], p, part)
                    self.ref[row[full]] -= 1
                    self.table[s][full], self.ref[p] = p, 1
                for j in range(first, held):
                    if j >= want or ref0[row[j]] != 1:
                        self.ref[row[j]] -= 1
                        self.table[s][j] = -1
                for j in take:
                    p = fresh.pop(0)
                    self.table[s][j], self.ref[p] = p, 1
            return len(take) + (1 if cow else 0), apply
        return self.serve(reqs, plan)

    def fork(self, reqs):  # (dst, src, len)
        pg = self.page

        def plan(r, ref0, table0):
            d, s, n = r
            if not (0 <= s < self.S and 0 <= n <= self.P * pg) or table0[d][0] >= 0:
                return None
            row, full, part = table0[s], n // pg, n % pg
            if any(not 0 <= row[j] < self.pages or ref0[row[j]] <= 0 for j in range(full + (part > 0))):
                return None

            def apply(fresh):
                for j in range(full):
                    self.table[d][j] = row[j]
                    self.ref[row[j]] += 1
                if part:
                    self.copy(row[full], fresh[0], part)
                    self.table[d][full], self.ref[fresh[0]] = fresh[0], 1
            return int(part > 0), apply
        return self.serve(reqs, plan)

    def compact(self):
        live = [p for p in range(self.pages) if self.ref[p] > 0]
        n = len(live)
        move = dict(zip([p for p in live if p >= n], [p for p in range(n) if self.ref[p] <= 0]))
        new = [move.get(p, p) if self.ref[p] > 0 else -1 for p in range(self.pages)]
        for a, b in move.items():
            self.copy(a, b, self.page)
            self.ref[b], self.ref[a] = self.ref[a], 0
        self.table = [[new[p] if 0 <= p < self.pages else p for p in row] for row in self.table]
        return new

    def check(self):
        assert self.dt.cpu().tolist() == self.table
        assert self.dr.cpu().tolist() == self.ref
        assert torch.equal(self.dk.cpu(), self.k) and torch.equal(self.dv.cpu(), self.v)


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32).cuda()


def do_resize(bsa, m, reqs, **kw):
    got = bsa.cache_resize(m.dt, m.dr, *(ints(r[i] for r in reqs) for i in range(3)), m.dk, m.dv, **kw)
    assert got.cpu().tolist() == m.resize(reqs), reqs
    m.check()


def do_fork(bsa, m, reqs):
    got = bsa.cache_fork(m.dt, m.dr, *(ints(r[i] for r in reqs) for i in (1, 0, 2)), m.dk, m.dv)
    assert got.cpu().tolist() == m.fork(reqs), reqs
    m.check()


def do_compact(bsa, m):
    got = bsa.cache_compact(m.dt, m.dr, m.dk, m.dv)
    assert got.cpu().tolist() == m.compact()
    m.check()


@pytest.mark.parametrize("seed,S,P,pages,layers,Hkv,page,D", [
    (0, 6, 5, 20, 2, 3, 64, 64), (1, 1, 1, 1, 1, 1, 128, 128), (2, 40, 9, 150, 1, 2, 64, 128),
    (3, 300, 33, 5000, 1, 1, 64, 64), (4, 12, 140, 900, 3, 1, 64, 64), (5, 1100, 4, 4200, 1, 1, 64, 64)])
def test_random_histories(bsa, seed, S, P, pages, layers, Hkv, page, D):
    """Grow, shrink, fork, free and compact in random order, bad and repeated
    requests among them, against the model after every call."""
    r = random.Random(seed)
    m = Model(S, P, pages, layers, Hkv, page, D, seed)
    for _ in range(14):
        n = r.choice([1, 2, 5, min(S + 3, 1300)])
        what = r.randrange(4)
        if what < 2:
            reqs = []
            for _ in range(n):
                s = r.randrange(-1, S + 1)
                have = m.held(s) * page if 0 <= s < S else 0
                keep = r.choice([0, have, r.randint(0, max(0, have)), have + 1])
                cap = r.choice([keep, keep, min(P * page, keep + r.randint(0, 3 * page)), r.randint(0, P * page + 5)])
                reqs.append((s, keep, cap))
            do_resize(bsa, m, reqs)
        elif what == 2:
            empty = [s for s in range(S) if m.held(s) == 0] or [0]
            reqs = []
            for _ in range(n):
                s = r.randrange(S)
                have = m.held(s) * page
                reqs.append((r.choice(empty + [r.randrange(-1, S + 1)]), s, r.choice([have, r.randint(0, have),
                                                                                    have + 1])))
            do_fork(bsa, m, reqs)
        else:
            do_compact(bsa, m)
    bsa.device_error()


@pytest.mark.parametrize("S,P,pages,n", [
    (3, 300, 16384, 3), (3, 300, 16385, 3), (4096, 2, 70, 12), (4097, 2, 70, 12), (2100, 2, 4300, 2048),
    (2100, 2, 4300, 2049)])
def test_up_to_what_one_cta_takes_and_beyond(bsa, S, P, pages, n):
    """The sizes where a request's check moves from one CTA to all of them."""
    r = random.Random(S * P + n)
    m = Model(S, P, pages, 1, 1, 64, 64, n)
    half = r.sample(range(S), n)
    do_resize(bsa, m, [(s, 0, r.randint(0, P * 64)) for s in half])
    # scatter what is free over the whole pool, up to its last page
    do_resize(bsa, m, [(s, 0, 0) for s in half[::2]] + [(half[-1], 0, 1)])
    last = next(s for s in range(S) if m.held(s) == 0)
    m.ref[pages - 1] += 1
    m.table[last][0] = pages - 1
    m.dr[pages - 1] += 1
    m.dt[last, 0] = pages - 1
    held = [s for s in range(S) if m.held(s)]
    empty = [s for s in range(S) if not m.held(s)]
    reqs = [(e, r.choice(held), r.randint(0, 64)) for e in empty]
    do_fork(bsa, m, (reqs * 3)[:n])
    do_compact(bsa, m)
    do_resize(bsa, m, [(s, 0, 0) for s in range(S)][:n])
    bsa.device_error()


def test_refusals_set_the_error_word(bsa):
    m = Model(4, 4, 6, 1, 1)
    do_resize(bsa, m, [(0, 0, 256), (1, 0, 100)])       # the whole pool
    assert bsa.device_error() == 0
    do_resize(bsa, m, [(2, 0, 1)])                      # empty
    assert bsa.device_error() == 64
    do_resize(bsa, m, [(0, 64, 64), (2, 0, 64)])        # what a call gives back, a later one takes
    assert bsa.device_error() == 64
    do_resize(bsa, m, [(2, 0, 64), (2, 0, 128)])        # the same sequence twice: the first
    assert bsa.device_error() == 64
    do_fork(bsa, m, [(3, 0, 64), (3, 1, 64)])           # the same destination twice
    assert bsa.device_error() == 64
    do_fork(bsa, m, [(3, 1, 64)])                       # a destination that holds pages
    assert bsa.device_error() == 64


def test_sharing_ends_where_writing_begins(bsa):
    """After a shrink into shared pages everything from `keep` on is the sequence's own."""
    m = Model(5, 6, 40, 2, 2)
    do_resize(bsa, m, [(0, 0, 5 * 64)])
    do_fork(bsa, m, [(1, 0, 320), (2, 0, 300), (3, 1, 129), (4, 0, 0)])
    assert bsa.device_error() == 64                     # 1 holds nothing when the call starts
    do_fork(bsa, m, [(3, 1, 129)])
    do_resize(bsa, m, [(1, 130, 384), (0, 64, 64)])     # both let go of the same pages
    do_resize(bsa, m, [(3, 128, 129), (2, 1, 1)])
    do_compact(bsa, m)
    for s in range(5):
        do_resize(bsa, m, [(s, 0, 0)])
    assert m.ref == [0] * 40 and bsa.device_error() == 0


def test_broken_tables_are_refused(bsa):
    m = Model(3, 3, 8, 1, 1)
    do_resize(bsa, m, [(0, 0, 192)])
    for bad in (99, 7):                                 # past the pool; a page that is free
        m.table[0][1] = bad
        m.dt[0, 1] = bad
        do_resize(bsa, m, [(0, 0, 0)])
        do_fork(bsa, m, [(1, 0, 128), (2, 0, 64)])
        assert bsa.device_error() == 64
        do_resize(bsa, m, [(2, 0, 0)])
    # entry 7 is free: it becomes -1.  Page 1 is still counted, so the three live pages stay where they are
    got = bsa.cache_compact(m.dt, m.dr, m.dk, m.dv)
    assert bsa.device_error() == 32 and m.dt[0].tolist() == [0, -1, 2] and got.tolist() == [0, 1, 2] + [-1] * 5


def test_streams_and_graphs(bsa):
    m = Model(4, 4, 12, 2, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    do_resize(bsa, m, [(0, 0, 200)], stream=s)
    dst, src, n, zero = ints([1, 2]), ints([0, 0]), ints([70, 130]), ints([0, 0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bsa.cache_resize(m.dt, m.dr, dst, zero, zero, m.dk, m.dv)
        got = bsa.cache_fork(m.dt, m.dr, src, dst, n, m.dk, m.dv)
    for _ in range(3):
        m.resize([(1, 0, 0), (2, 0, 0)])
        want = m.fork([(1, 0, 70), (2, 0, 130)])
        g.replay()
        assert got.tolist() == want
        m.check()
    assert bsa.device_error() == 0


def test_no_requests(bsa):
    m = Model(2, 2, 4, 1, 1)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    assert bsa.cache_resize(m.dt, m.dr, e, e, e, m.dk, m.dv).numel() == 0
    assert bsa.cache_fork(m.dt, m.dr, e, e, e, m.dk, m.dv).numel() == 0
    m.check()


# ------------------------------------------------------------ accept
@pytest.mark.parametrize("layers,S,T,Hkv,page,D", [(1, 1, 1, 1, 64, 64), (1, 7, 5, 3, 64, 128), (3, 20, 16, 2, 128, 64),
                                                   (2, 9, 64, 1, 64, 128), (1, 300, 8, 8, 128, 128)])
def test_accept(bsa, layers, S, T, Hkv, page, D):
    r = random.Random(S * T)
    ctx = [r.choice([0, 1, page - 1, page, r.randint(0, 3 * page)]) for _ in range(S)]
    m = Model(S, 6, S * 6, layers, Hkv, page, D, S)
    m.resize([(s, 0, ctx[s] + T) for s in range(S)])
    dt = torch.tensor(m.table, dtype=torch.int32).cuda()
    acc, na = torch.full((S, T), -9, dtype=torch.int32), []
    for s in range(S):
        k = r.randint(0, T)
        acc[s, :k] = torch.tensor(sorted(r.sample(range(T), k)), dtype=torch.int32)
        na.append(k)
    new = bsa.cache_accept(m.dk, m.dv, dt, ints(ctx), acc.cuda(), ints(na))
    assert new.tolist() == [c + n for c, n in zip(ctx, na)]
    for t in (m.k, m.v):
        t = t if t.dim() == 5 else t[None]
        for s in range(S):
            at = lambda x: (m.table[s][x // page], x % page)
            rows = [t[:, at(ctx[s] + int(acc[s, i]))[0], :, at(ctx[s] + int(acc[s, i]))[1]].clone()
                    for i in range(na[s])]
            for i, row in enumerate(rows):
                p, q = at(ctx[s] + i)
                t[:, p, :, q] = row
    assert torch.equal(m.dk.cpu(), m.k) and torch.equal(m.dv.cpu(), m.v)
    assert bsa.device_error() == 0


def test_accept_refuses_bad_lists(bsa):
    """Not increasing, out of range, too many, a missing page: reported, rows and length kept."""
    m = Model(7, 2, 14, 1, 1)
    m.resize([(s, 0, 128) for s in range(6)] + [(6, 0, 64)])
    dt = torch.tensor(m.table, dtype=torch.int32).cuda()
    acc = ints([1, 1, 0, 2, 0, 0, 0, 4, 0, -1, 2, 0, 0, 2, 3, 1, 3, 0, 1, 2, 3]).reshape(7, 3)
    na = ints([2, 2, 2, 2, 4, -1, 2])
    acc[1] = ints([2, 1, 0])
    new = bsa.cache_accept(m.dk, m.dv, dt, ints([60] * 6 + [62]), acc.clamp(max=9), na)
    assert bsa.device_error() == 32
    # 0: 1,1 repeats; 1: decreases; 2: 0, 4 out of range; 3: -1 first; 4: four of three; 5: negative; 6: slot 64 has no page
    assert new.tolist() == [60, 60, 60, 60, 60, 60, 62]
    assert torch.equal(m.dk.cpu(), m.k) and torch.equal(m.dv.cpu(), m.v)
    # others in the same call go ahead
    acc[0] = ints([1, 2, 0])
    new = bsa.cache_accept(m.dk, m.dv, dt, ints([60] * 6 + [62]), acc, na)
    assert bsa.device_error() == 32 and new.tolist()[0] == 62
    p = m.table[0][0]
    for d, t in ((m.dk, m.k), (m.dv, m.v)):
        assert torch.equal(d[p, :, 60:62].cpu(), t[p, :, 61:63])
