"""Caches of 8-bit rows: appending, reading back, and the page calls.

Tolerance of an appended row, derived before the first run: the normed and
rotated values are within 2^-19 of their size (test_gpu_rope's angles and fp32
steps) before the one rounding to a code.  A code is the nearest one, so a value
that lies within that of a border between two codes may take either: |held - y|
<= 2^-4 |y| (half a step) + 2^-18 max |y|, or half of the smallest code's step,
2^-10 * 2^e.  The scale may differ only where max |y| lies within 2^-18 of
448 * 2^e.
"""

import math

import pytest
import torch

from paged_reference import E4M3, E8M0, Cache, e4m3_values, quantise, values

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


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rotated(y, w, pos, inv_freq, gain, interleaved):
    y = y.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.double()
    rd = 2 * len(inv_freq)
    ang = pos.double()[:, None] * inv_freq
    c, s = (gain * ang.cos())[:, None], (gain * ang.sin())[:, None]
    out = y.clone()
    a, b = (y[..., 0:rd:2], y[..., 1:rd:2]) if interleaved else (y[..., :rd // 2], y[..., rd // 2:rd])
    x, z = a * c - b * s, b * c + a * s
    if interleaved:
        out[..., 0:rd:2], out[..., 1:rd:2] = x, z
    else:
        out[..., :rd // 2], out[..., rd // 2:rd] = x, z
    return out


def empty_pools(n_pages, Hkv, page, D):
    k = torch.full((n_pages, Hkv, page, D), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((n_pages, Hkv, page), 77, dtype=torch.uint8, device="cuda")
    return k, k.clone(), s, s.clone()


def check_rows(codes, scales, y):
    """Held rows (uint8 codes and scale bytes) against 64-bit values y."""
    want_codes, want = quantise(y)
    top = y.abs().amax(-1)
    differ = want != scales
    if differ.any():
        e = scales[differ].double() - 127
        edge = torch.minimum((top[differ] / (448 * torch.pow(2.0, e)) - 1).abs(),
                             (top[differ] / (448 * torch.pow(2.0, e - 1)) - 1).abs())
        assert (edge < 2.0 ** -18).all()
    held, e = values(codes, scales), torch.pow(2.0, scales.double() - 127)[..., None]
    tol = torch.maximum(y.abs() * 2.0 ** -4, e * 2.0 ** -10) + top[..., None] * 2.0 ** -18
    assert ((held - y).abs() <= tol).all()
    return float((codes != want_codes).double().mean())


# ------------------------------------------------------------ appending
@pytest.mark.parametrize("D,page", [(64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm,rd", [(True, 64), (False, 32), (True, 16)])
@pytest.mark.parametrize("N", [1, 37, 700])
def test_append(bsa, D, page, interleaved, norm, rd, N):
    g = torch.Generator().manual_seed(N + D)
    Hq, Hkv = 6, 3
    x = (torch.randn(N, Hq + 2 * Hkv, D, generator=g) * torch.exp(torch.randn(N, Hq + 2 * Hkv, 1, generator=g) * 2)).bfloat16()
    w = [1 + 0.2 * torch.randn(D, generator=g) for _ in range(2)] if norm else [None, None]
    B, P = 3, 6
    table = torch.randperm(B * P, generator=g).int().reshape(B, P)
    where = torch.randperm(B * P * page, generator=g)[:N]
    seq, slot = (where // (P * page)).int(), (where % (P * page)).int()
    kc, vc, ks, vs = empty_pools(B * P + 2, Hkv, page, D)
    k0, s0 = kc.clone(), ks.clone()
    inv = bsa.rope_inv_freq(rd)
    xd, wd = x.cuda(), [None if t is None else t.cuda() for t in w]
    zq = bsa.cache_append(xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], kc.view(E4M3), vc.view(E4M3), table.cuda(),
                          seq.cuda(), slot.cuda(), inv, q_weight=wd[0], k_weight=wd[1], interleaved=interleaved,
                          k_scale=ks.view(E8M0), v_scale=vs.view(E8M0))
    assert bsa.device_error() == 0
    # the queries are those of the bf16 cache's call, bit for bit
    kb, vb = (torch.zeros(B * P + 2, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    zq2 = bsa.cache_append(xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], kb, vb, table.cuda(), seq.cuda(), slot.cuda(),
                           inv, q_weight=wd[0], k_weight=wd[1], interleaved=interleaved)
    assert torch.equal(zq, zq2)
    pg, at = table[seq.long(), slot.long() // page].long(), slot.long() % page
    off = check_rows(kc.cpu()[pg, :, at], ks.cpu()[pg, :, at],
                     rotated(x[:, Hq:Hq + Hkv], w[1], slot, inv.cpu(), 1.0, interleaved))
    assert off < 1e-3  # only codes within 2^-18 of a border may be others
    y = x[:, Hq + Hkv:].double()  # values are only moved: exactly the nearest codes
    codes, scales = quantise(y)
    assert torch.equal(vc.cpu()[pg, :, at], codes) and torch.equal(vs.cpu()[pg, :, at], scales)
    # nothing else was written
    for pool, was in ((kc, k0), (vc, k0), (ks, s0), (vs, s0)):
        rest = torch.ones(pool.shape[0], page, dtype=torch.bool)
        rest[pg, at] = False
        a, b = pool.cpu().transpose(1, 2)[rest], was.cpu().transpose(1, 2)[rest]
        assert torch.equal(a, b)


def test_append_extremes(bsa):
    """Rows of zeros, of one value, at the borders of the scales, at the types' ends; infinities and NaN."""
    D = 64
    vals = [0.0, 448.0, 450.0, 2.0 ** -9, 3.5, 1.75 * 2.0 ** -20, 2.0 ** -126, 2.0 ** -133, 2.0 ** 120, 3.3e38, 1.0 / 3, 57344.0]
    rows = torch.zeros(len(vals) + 3, 3, D)
    for i, x in enumerate(vals):
        rows[i, 1:] = torch.linspace(-1, 1, D) * 0
        rows[i, 1:, ::3] = x
        rows[i, 1:, 1::3] = -x / 2
    rows[-3, 1:, 5], rows[-2, 1:, 7], rows[-1, 1:, 9] = math.inf, -math.inf, math.nan
    rows[-3:, 1:, 0] = 1.0
    x = rows.bfloat16()
    n = x.shape[0]
    kc, vc, ks, vs = empty_pools(1, 1, 64, D)
    bsa.cache_append(x[:, :1].cuda(), x[:, 1:2].cuda(), x[:, 2:].cuda(), kc.view(E4M3), vc.view(E4M3),
                     i32([[0]]), i32([0] * n), torch.arange(n, dtype=torch.int32, device="cuda"), k_scale=ks.view(E8M0),
                     v_scale=vs.view(E8M0))
    assert bsa.device_error() == 0
    m = len(vals)
    codes, scales = quantise(x[:m, 2].double())
    for pool, sc in ((kc, ks), (vc, vs)):
        assert torch.equal(pool.cpu()[0, 0, :m], codes) and torch.equal(sc.cpu()[0, 0, :m], scales)
        assert sc.cpu()[0, 0, m:m + 2].tolist() == [118 + 127] * 2
        assert pool.cpu()[0, 0, m, 5] == 0x7E and pool.cpu()[0, 0, m + 1, 7] == 0xFE  # +-448
        assert pool.cpu()[0, 0, m + 2, 9] & 0x7F == 0x7F


def test_append_padding_and_bad_places(bsa):
    D, page = 128, 64
    x = torch.randn(5, 3, D).bfloat16().cuda()
    kc, vc, ks, vs = empty_pools(3, 1, page, D)
    was = [t.clone() for t in (kc, vc, ks, vs)]
    table = i32([[0, -1], [7, 1]])
    q = bsa.cache_append(x[:, :1], x[:, 1:2], x[:, 2:], kc.view(E4M3), vc.view(E4M3), table, i32([-1, 0, 1, 5, 0]),
                         i32([3, 64, 0, 0, -1]), k_scale=ks.view(E8M0), v_scale=vs.view(E8M0))
    assert bsa.device_error() == 32
    for a, b in zip((kc, vc, ks, vs), was):
        assert torch.equal(a, b)
    assert q.shape == (5, 1, D)


# ------------------------------------------------------------ reading back
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("D,page,rep", [(64, 64, 1), (64, 128, 3), (128, 64, 2), (128, 128, 1)])
@pytest.mark.parametrize("n", [1, 63, 64, 65, 500])
def test_read(bsa, q8, D, page, rep, n):
    lens = [400, 70, 1, 600]
    c = Cache(lens, 2, D, page, q8, seed=n)
    k, v, table, sc = c.device()
    seq = [3, -1, 0, 1, 3]
    first = [0, 0, 5, 10, 100]
    want = [min(n, 600), n, min(n, 300), min(n, 60), min(n, 0)]
    ok, ov = bsa.cache_read(k, v, table, i32(seq), i32(want), n, first=i32(first), kv_repeat=rep, **sc)
    assert bsa.device_error() == 0
    assert ok.shape == (5, 2 * rep, n, D)
    for i, (b, f, m) in enumerate(zip(seq, first, want)):
        m = 0 if b < 0 else m
        assert (ok[i, :, m:] == 0).all() and (ov[i, :, m:] == 0).all()
        for h in range(2 * rep):
            K, V = c.rows(b, h // rep, torch.arange(f, f + m))
            assert torch.equal(ok[i, h, :m].cpu().double(), K) and torch.equal(ov[i, h, :m].cpu().double(), V)


def test_read_every_code_and_scale(bsa):
    codes = torch.arange(256, dtype=torch.uint8).reshape(4, 64).repeat(16, 1)
    scales = torch.tensor([27, 60, 100, 127, 128, 134, 135, 180, 245], dtype=torch.uint8)
    k = codes.reshape(1, 1, 64, 64).cuda()
    s = scales.repeat(8)[:64].reshape(1, 1, 64).cuda()
    ok, ov = bsa.cache_read(k, k, i32([[0]]), i32([0]), None, 64, k_scale=s, v_scale=s)
    want = values(codes, s.cpu()[0, 0])
    for o in (ok, ov):
        got = o[0, 0].cpu().double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


def test_read_reports_what_is_not_there(bsa):
    c = Cache([200, 100], 1, 64, 64, False)
    k, v, table, _ = c.device()
    for seq, first, n in (([2], [0], 8), ([0], [-1], 8), ([0], [250], 8), ([0], [2 ** 31 - 1], 8), ([1], [120], 20)):
        ok, ov = bsa.cache_read(k, v, table, i32(seq), None, n, first=i32(first))
        assert bsa.device_error() == 32
        # what lies in a page (of 4 and 2) comes back, whether or not it was written
        m = 0 if seq == [2] or first == [-1] else max(0, min(n, {0: 256, 1: 128}[seq[0]] - first[0]))
        assert (ok[0, 0, m:] == 0).all() and torch.isnan(ok[0, 0, :m]).all()
    bsa.cache_read(k, v, table, i32([0]), i32([9]), 8)
    assert bsa.device_error() == 32
    ok, _ = bsa.cache_read(k, v, table, i32([]), None, 8)
    assert ok.shape == (0, 1, 8, 64)
    ok, _ = bsa.cache_read(k, v, table, i32([0]), None, 0)
    assert ok.shape == (1, 1, 0, 64) and bsa.device_error() == 0


# ------------------------------------------------------------ pages
def layered(L, n_pages, Hkv, page, D, seed):
    g = torch.Generator().manual_seed(seed)
    pools = [torch.randint(0, 256, (L, n_pages, Hkv, page, D), generator=g).to(torch.uint8) for _ in range(2)]
    scales = [torch.randint(0, 256, (L, n_pages, Hkv, page), generator=g).to(torch.uint8) for _ in range(2)]
    return pools, scales


@pytest.mark.parametrize("D,page", [(64, 64), (128, 64), (128, 128)])
def test_fork_and_resize_move_codes_and_scales(bsa, D, page):
    L, P, Hkv = 3, 12, 2
    pools, scales = layered(L, P, Hkv, page, D, 1)
    table = torch.full((4, 4), -1, dtype=torch.int32)
    table[0, :3] = torch.tensor([5, 2, 9], dtype=torch.int32)
    ref = torch.zeros(P, dtype=torch.int32)
    ref[[5, 2, 9]] = 1
    kc, vc, ks, vs, td, rd = (t.cuda() for t in (*pools, *scales, table, ref))
    kw = dict(k_scale=ks, v_scale=vs)
    n = 2 * page + 37
    got = bsa.cache_fork(td, rd, i32([0, 0]), i32([1, 2]), i32([n, page]), kc, vc, **kw)
    assert got.tolist() == [1, 1] and td[1].tolist() == [5, 2, 0, -1] and td[2].tolist() == [5, -1, -1, -1]
    for dst, src in ((kc, pools[0]), (vc, pools[1]), (ks, scales[0]), (vs, scales[1])):
        d = dst.cpu()
        assert torch.equal(d[:, 0, :, :37], src[:, 9, :, :37])
        assert torch.equal(d[:, 0, :, 37:], src[:, 0, :, 37:]) and torch.equal(d[:, 1:], src[:, 1:])
    # sequence 1 keeps page + 5 slots: the shared page 2 is copied for it
    got = bsa.cache_resize(td, rd, i32([1]), i32([page + 5]), i32([page + 50]), kc, vc, **kw)
    assert got.tolist() == [1]
    new = int(td[1, 1])
    assert new not in (5, 2, 9) and td[1].tolist()[2:] == [-1, -1]
    for dst, src in ((kc, pools[0]), (vc, pools[1]), (ks, scales[0]), (vs, scales[1])):
        assert torch.equal(dst.cpu()[:, new, :, :5], src[:, 2, :, :5])
    assert bsa.device_error() == 0


def test_compact_moves_codes_and_scales(bsa):
    L, P, Hkv, page, D = 2, 10, 3, 64, 64
    pools, scales = layered(L, P, Hkv, page, D, 2)
    table = torch.tensor([[9, 3, -1], [7, 3, 8]], dtype=torch.int32)
    ref = torch.zeros(P, dtype=torch.int32)
    for x in (9, 3, 7, 3, 8):
        ref[x] += 1
    kc, vc, ks, vs, td, rd = (t.cuda() for t in (*pools, *scales, table, ref))
    new = bsa.cache_compact(td, rd, kc, vc, k_scale=ks, v_scale=vs).cpu()
    assert bsa.device_error() == 0 and sorted(x for x in new.tolist() if x >= 0) == [0, 1, 2, 3]
    for old in (9, 3, 7, 8):
        for dst, src in ((kc, pools[0]), (vc, pools[1]), (ks, scales[0]), (vs, scales[1])):
            assert torch.equal(dst.cpu()[:, int(new[old])], src[:, old])
    assert torch.equal(td.cpu(), torch.where(table >= 0, new[table.clamp(min=0).long()], -1))


@pytest.mark.parametrize("D,Hkv", [(64, 1), (128, 8), (64, 300)])
def test_accept_moves_codes_and_scales(bsa, D, Hkv):
    L, page, T = 2, 64, 9
    pools, scales = layered(L, 6, Hkv, page, D, 3)
    table = torch.tensor([[4, 1], [0, 2]], dtype=torch.int32)
    ctx, acc, na = [60, 10], torch.zeros(2, T, dtype=torch.int32), [4, 2]
    acc[0, :4] = torch.tensor([0, 3, 5, 8], dtype=torch.int32)
    acc[1, :2] = torch.tensor([1, 2], dtype=torch.int32)
    kc, vc, ks, vs = (t.cuda() for t in (*pools, *scales))
    new = bsa.cache_accept(kc, vc, table.cuda(), i32(ctx), acc.cuda(), i32(na), k_scale=ks, v_scale=vs)
    assert new.tolist() == [64, 12] and bsa.device_error() == 0
    for dst, src in ((kc, pools[0]), (vc, pools[1]), (ks, scales[0]), (vs, scales[1])):
        want = src.clone()
        for b in range(2):
            for i in range(na[b]):
                a, z = ctx[b] + int(acc[b, i]), ctx[b] + i
                want[:, table[b, z // page].item(), :, z % page] = src[:, table[b, a // page].item(), :, a % page]
        assert torch.equal(dst.cpu(), want)


# ------------------------------------------------------------ the calls in a row
@pytest.mark.parametrize("q8", [False, True])
def test_prompt_in_chunks_then_decoding(bsa, q8):
    """A prompt appended and attended to in three chunks, then decoded: what each
    call returns is the attention of the rows that the cache holds; the prompt read
    back gives the block-sparse forward the same rows."""
    g = torch.Generator().manual_seed(5)
    Hq, Hkv, D, page, S = 8, 2, 128, 64, 3
    P = 8
    kc, vc = (torch.zeros(P + 1, Hkv, page, D, dtype=E4M3 if q8 else torch.bfloat16, device="cuda") for _ in range(2))
    sc = {}
    if q8:
        ks = torch.zeros(P + 1, Hkv, page, dtype=torch.uint8, device="cuda")
        sc = dict(k_scale=ks.view(E8M0), v_scale=ks.clone().view(E8M0))
    table, ref = torch.full((1, P), -1, dtype=torch.int32, device="cuda"), torch.zeros(P + 1, dtype=torch.int32, device="cuda")
    inv, w = bsa.rope_inv_freq(D), torch.ones(D, device="cuda")
    at = 0
    outs = []
    for n in (150, 100, 6, 1, 1):
        assert bsa.cache_resize(table, ref, i32([0]), i32([at]), i32([at + n]), kc, vc, **sc).tolist() == [1]
        x = torch.randn(n, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
        slots = torch.arange(at, at + n, dtype=torch.int32, device="cuda")
        q = bsa.cache_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kc, vc, table, torch.zeros_like(slots), slots,
                             inv, q_weight=w, k_weight=w, **sc)
        o, l = bsa.chunk_attention(q, kc, vc, table, i32([at]), q_ptr=i32([0, n]), **sc)
        outs.append((at, n, q, o, l))
        at += n
    assert bsa.device_error() == 0
    k, v = bsa.cache_read(kc, vc, table, i32([0]), i32([at]), 384, kv_repeat=Hq // Hkv, **sc)
    K, V = (t[0, :, :at].cpu().double() for t in (k, v))
    for start, n, q, o, l in outs:
        S_ = torch.einsum("thd,hsd->ths", q.cpu().double(), K[:, :start + n]) / math.sqrt(D)
        S_ = S_.masked_fill(torch.arange(start + n)[None, None] > torch.arange(start, start + n)[:, None, None], -math.inf)
        lse = torch.logsumexp(S_, -1)
        O = torch.einsum("ths,hsd->thd", torch.exp(S_ - lse[..., None]), V[:, :start + n])
        assert (l.cpu().double() - lse).abs().max() < 1e-4
        assert (o.cpu().double() - O).abs().max() < 2.0 ** -6 * V.abs().max()
    # the forward over the read rows (the whole prompt's queries, dense blocks, causal) gives the same outputs
    q = torch.zeros(1, Hq, 384, D, dtype=torch.bfloat16, device="cuda")
    for start, n, qc, _, _ in outs:
        q[0, :, start:start + n] = qc.transpose(0, 1)
    pat = bsa.Pattern(6, 6, 0, causal=True)
    rp, ci = bsa.build_mask_csr(pat, 1, Hq, device="cuda")
    of, lf = bsa.forward(q, k, v, rp, ci, 64, causal=True)
    for start, n, _, o, l in outs:
        assert (lf[0, :, start:start + n].T - l).abs().max() < 1e-3
        assert (of[0, :, start:start + n].transpose(0, 1).float() - o.float()).abs().max() < 2.0 ** -5 * V.abs().max()
