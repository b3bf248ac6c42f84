"""qk_norm_rope, its gradients and cache_append against the definition in 64
bits (numpy), on one GPU.

Tolerances, derived before the first run.  One output rounding: |ref| * 2^-8
at most (bf16 half step).  The fp32 part before it: the angle is good to 2^-20
(include/bsa.h), a few fp32 roundings of 2^-24 on the norm, both relative to
the pair, whose size is at most sqrt(2) * the row's largest normed value:
2^-18 * that.  Weight gradients (fp32) are sums over rows of dy * x * r with
the same relative error per term, plus at most 2^-24 per addition along the
longest chain of additions (rows a lane adds in turn, then 32 + 12 levels),
relative to the sum of the terms' magnitudes."""

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


def f64(t):
    return t.detach().cpu().double().numpy()


def pairs_of(rd, il):
    i = np.arange(rd // 2)
    return (2 * i, 2 * i + 1) if il else (i, i + rd // 2)


def ref_rows(x, w, pos, freq, eps, gain, il):
    """x [..., H, D] (float64), pos [...]: normed and rotated rows."""
    y = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    z = y.copy()
    if freq is not None:
        a, b = pairs_of(2 * len(freq), il)
        ang = pos[..., None].astype(np.float64) * freq
        c, s = np.cos(ang)[..., None, :], np.sin(ang)[..., None, :]
        z[..., a] = gain * (y[..., a] * c - y[..., b] * s)
        z[..., b] = gain * (y[..., b] * c + y[..., a] * s)
    return y, z


def ref_grad(x, dz, w, pos, freq, eps, gain, il):
    """Gradients of sum(z * dz) for x [B,N,H,D] and w; and the size of their terms."""
    dy = dz.copy()
    if freq is not None:
        a, b = pairs_of(2 * len(freq), il)
        ang = pos[..., None].astype(np.float64) * freq
        c, s = np.cos(ang)[..., None, :], np.sin(ang)[..., None, :]
        dy[..., a] = gain * (dz[..., a] * c + dz[..., b] * s)
        dy[..., b] = gain * (dz[..., b] * c - dz[..., a] * s)
    if w is None:
        return dy, None, np.abs(dy).max(-1, keepdims=True), None
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = dy * w
    m = (g * x).mean(-1, keepdims=True)
    dx = r * g - x * r ** 3 * m
    size = r * np.abs(g).max(-1, keepdims=True) + np.abs(x).max(-1, keepdims=True) * r ** 3 * np.abs(g * x).mean(
        -1, keepdims=True)
    t = dy * x * r
    big = np.abs(dy).max(-1, keepdims=True) * np.abs(x) * r  # a term's rotation error goes with its pair
    return dx, t.sum((0, 1, 2)), size, big.sum((0, 1, 2))


def within(got, ref, size, what):
    err = np.abs(got - ref)
    tol = np.abs(ref) * 2.0 ** -8 + size * 2.0 ** -18 + 1e-38
    assert np.isfinite(got).all(), what
    assert (err <= tol).all(), "%s: %.3g over the tolerance" % (what, (err / tol).max())


CASES = [  # B, N, Hq, Hkv, rep, D, rd, interleaved, norm, how positions come
    (1, 1, 1, 1, 1, 64, 64, False, "qk", None),
    (1, 1, 3, 1, 3, 128, 128, True, "qk", "far"),
    (2, 7, 5, 5, 1, 64, 16, False, "q", "batch"),
    (1, 33, 8, 2, 4, 128, 32, True, "k", "row"),
    (3, 65, 4, 2, 1, 128, 112, False, "qk", "far"),
    (2, 127, 6, 3, 2, 64, 48, True, "", "negative"),
    (1, 1000, 16, 4, 1, 128, 64, False, "qk", None),
    (2, 515, 7, 1, 7, 64, 0, False, "qk", None),
    (1, 4099, 20, 5, 4, 64, 64, True, "qk", "row"),
    (1, 2048, 9, 9, 1, 128, 128, False, "", None),
]


def make(case, seed=0):
    B, N, Hq, Hkv, rep, D, rd, il, norm, how = case
    g = torch.Generator().manual_seed(seed + N)
    qkv = torch.randn(B, N, Hq + 2 * Hkv, D, generator=g).bfloat16()
    qw = (1 + 0.3 * torch.randn(D, generator=g)) if "q" in norm else None
    kw = (1 + 0.3 * torch.randn(D, generator=g)) if "k" in norm else None
    freq = 10000.0 ** (-2 * torch.arange(rd // 2, dtype=torch.float64) / rd) if rd else None
    pos = None
    if how == "row":
        pos = torch.randint(0, 200000, (N,), generator=g, dtype=torch.int32)
    elif how == "batch":
        pos = torch.randint(0, 5000, (B, N), generator=g, dtype=torch.int32)
    elif how == "far":
        pos = torch.randint(2 ** 30, 2 ** 31 - 1, (B, N), generator=g, dtype=torch.int64).int()
    elif how == "negative":
        pos = torch.randint(-100000, 0, (B, N), generator=g, dtype=torch.int32)
    p = np.broadcast_to(np.arange(N) if pos is None else pos.numpy(), (B, N))
    return qkv, qw, kw, freq, pos, p


def dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(bsa, case):
    B, N, Hq, Hkv, rep, D, rd, il, norm, how = case
    qkv, qw, kw, freq, pos, p = make(case)
    x, dqw, dkw, dfreq, dpos = dev(qkv, qw, kw, freq, pos)
    zq, zk, zv = bsa.qk_norm_rope(x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], dfreq, positions=dpos,
                                  q_weight=dqw, k_weight=dkw, eps=1e-5, gain=1.25, interleaved=il, kv_repeat=rep)
    X = f64(qkv)
    fr = None if freq is None else freq.numpy()
    for got, lo, hi, w, r in ((zq, 0, Hq, qw, 1), (zk, Hq, Hq + Hkv, kw, rep)):
        y, z = ref_rows(X[:, :, lo:hi], None if w is None else f64(w), p, fr, 1e-5, 1.25, il)
        z, y = (np.repeat(t.transpose(0, 2, 1, 3), r, axis=1) for t in (z, y))
        within(f64(got), z, 2 * np.abs(y).max(-1, keepdims=True), "q" if lo == 0 else "k")
    v = X[:, :, Hq + Hkv:].transpose(0, 2, 1, 3).repeat(rep, axis=1)
    np.testing.assert_array_equal(f64(zv), v)
    assert bsa.device_error() == 0


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(bsa, case):
    B, N, Hq, Hkv, rep, D, rd, il, norm, how = case
    qkv, qw, kw, freq, pos, p = make(case, 50)
    g = torch.Generator().manual_seed(7)
    dz = [torch.randn(B, H, N, D, generator=g).bfloat16() for H in (Hq, Hkv * rep, Hkv * rep)]
    x, dqw, dkw, dfreq, dpos, *ddz = dev(qkv, qw, kw, freq, pos, *dz)
    gx = torch.full((B, N, Hq + 2 * Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = (gx[:, :, :Hq], gx[:, :, Hq:Hq + Hkv], gx[:, :, Hq + Hkv:])
    *_, gqw, gkw = bsa.qk_norm_rope_backward(*ddz, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], dfreq, positions=dpos,
                                             q_weight=dqw, k_weight=dkw, eps=1e-5, gain=0.75, interleaved=il,
                                             kv_repeat=rep, out=out)
    X, fr = f64(qkv), None if freq is None else freq.numpy()
    for got, gw, lo, hi, w, r, d in ((out[0], gqw, 0, Hq, qw, 1, dz[0]), (out[1], gkw, Hq, Hq + Hkv, kw, rep, dz[1])):
        d = f64(d).reshape(B, hi - lo, r, N, D)
        D1 = d.sum(2).transpose(0, 2, 1, 3)
        dx, dw, size, terms = ref_grad(X[:, :, lo:hi], D1, None if w is None else f64(w), p, fr, 1e-5, 0.75, il)
        within(f64(got), dx, 4 * size, "q" if lo == 0 else "k")
        assert (gw is None) == (w is None)
        if w is not None:
            chain = B * N * (hi - lo) / 8 + 44
            tol = terms * 2 * (2.0 ** -18 + chain * 2.0 ** -24)
            assert (np.abs(f64(gw) - dw) <= tol).all()
    gv = f64(dz[2]).reshape(B, Hkv, rep, N, D).sum(2).transpose(0, 2, 1, 3)
    within(f64(out[2]), gv, np.abs(f64(dz[2])).max(), "v")
    assert bsa.device_error() == 0


def test_gradient_by_differences(bsa):
    """The formula's gradient, which the kernel is compared with above, against
    central differences of the 64-bit forward."""
    case = (1, 3, 2, 2, 1, 64, 32, True, "qk", "row")
    qkv, qw, kw, freq, pos, p = make(case)
    x, w = f64(qkv)[:, :, :2], f64(qw)
    rng = np.random.default_rng(0)
    dz = rng.standard_normal(x.shape)
    dx, dw, _, _ = ref_grad(x, dz, w, p, freq.numpy(), 1e-5, 1.3, True)
    f = lambda x, w: (ref_rows(x, w, p, freq.numpy(), 1e-5, 1.3, True)[1] * dz).sum()
    h = 1e-5  # truncation ~ h^2, rounding ~ 1e-16 * |f| / h ~ 1e-9
    for _ in range(20):
        i = tuple(rng.integers(0, n) for n in x.shape)
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-6
        j = rng.integers(0, 64)
        ew = np.zeros(64)
        ew[j] = h
        assert abs((f(x, w + ew) - f(x, w - ew)) / (2 * h) - dw[j]) < 1e-6


def test_position_zero_and_values_are_exact(bsa):
    """Without a norm, position 0 and the values past rotary_dim come through bit for bit."""
    x = torch.randn(1, 50, 6, 128, device="cuda").bfloat16()
    f = bsa.rope_inv_freq(64)
    z = torch.zeros(50, dtype=torch.int32, device="cuda")
    q, k, v = bsa.qk_norm_rope(x[:, :, :2], x[:, :, 2:4], x[:, :, 4:], f, positions=z)
    for got, lo in ((q, 0), (k, 2), (v, 4)):
        assert torch.equal(got, x[:, :, lo:lo + 2].transpose(1, 2))
    q, k, _ = bsa.qk_norm_rope(x[:, :, :2], x[:, :, 2:4], None, f)
    assert torch.equal(q[..., 64:], x[:, :, :2].transpose(1, 2)[..., 64:])


def test_no_tokens(bsa):
    x = torch.zeros(2, 0, 4, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda")
    q, k, v = bsa.qk_norm_rope(x, x, x, None, q_weight=w)
    assert q.shape == (2, 4, 0, 64) and v.shape == k.shape == q.shape
    gq, gk, gv, gw, gkw = bsa.qk_norm_rope_backward(q, k, v, x, x, None, q_weight=w)
    assert gq.shape == x.shape and gkw is None and torch.equal(gw, torch.zeros_like(w))


def test_special_values_stay_in_their_row(bsa):
    x = torch.randn(1, 40, 4, 64, device="cuda").bfloat16()
    w, f = torch.ones(64, device="cuda"), bsa.rope_inv_freq(64)
    good = bsa.qk_norm_rope(x, x, None, f, q_weight=w, k_weight=w)[0]
    y = x.clone()
    y[0, 3, 1, 5] = float("nan")
    y[0, 9, 2, 7] = float("inf")
    y[0, 11, 0] = 0  # a row of zeros normalises to zeros
    bad = bsa.qk_norm_rope(y, x, None, f, q_weight=w, k_weight=w)[0]
    assert bad[0, 1, 3].isnan().all() and bad[0, 2, 9].isnan().any() and (bad[0, 0, 11] == 0).all()
    keep = torch.ones(4, 40, dtype=torch.bool, device="cuda")
    keep[1, 3] = keep[2, 9] = keep[0, 11] = False
    assert torch.equal(bad[0][keep], good[0][keep])
    # eps = 0 and a zero row: that row is not a number, the weight's gradient of the other rows' kind too,
    # but rows that a tile does not hold must not leak into it
    g = torch.randn(1, 4, 40, 64, device="cuda").bfloat16()
    _, _, _, gw, _ = bsa.qk_norm_rope_backward(g, g, None, x, x, f, q_weight=w, k_weight=w, eps=0.0)
    assert gw.isfinite().all()


def test_streams_graphs_and_repeats(bsa):
    """Another stream, a captured pair of forward and backward replayed on new
    contents while eager calls run between, and equal bits every time."""
    case = (1, 777, 8, 2, 4, 128, 128, False, "qk", None)
    qkv, qw, kw, freq, pos, p = make(case)
    x, dqw, dkw, f = dev(qkv, qw, kw, freq)
    args = dict(q_weight=dqw, k_weight=dkw, kv_repeat=4)

    def both(stream=None):
        z = bsa.qk_norm_rope(x[:, :, :8], x[:, :, 8:10], x[:, :, 10:], f, stream=stream, **args)
        return z, bsa.qk_norm_rope_backward(*z, x[:, :, :8], x[:, :, 8:10], f, stream=stream, **args)

    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = both(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = both()
    x.copy_(qkv.cuda() * 2)
    graph.replay()
    other = both()
    flat = lambda r: [t for part in r for t in part]
    for a, b in zip(flat(third), flat(other)):
        assert torch.equal(a, b)
    x.copy_(qkv)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(flat(first), flat(second), flat(third)):
        assert torch.equal(a, b) and torch.equal(a, c)


# ------------------------------------------------------------ append
@pytest.mark.parametrize("tokens,Hq,Hkv,D,page,rd,il,norm,strided", [
    (1, 16, 16, 128, 128, 128, False, "qk", False), (1, 1, 1, 64, 64, 64, True, "", True),
    (5, 6, 3, 64, 128, 32, True, "q", True), (37, 8, 2, 128, 64, 64, False, "qk", True),
    (300, 10, 2, 128, 128, 16, True, "k", False), (2048, 32, 8, 64, 64, 64, False, "", True)])
def test_append(bsa, tokens, Hq, Hkv, D, page, rd, il, norm, strided):
    g = torch.Generator().manual_seed(tokens)
    S, maxp = 9, 6
    n_pages = S * maxp + 2
    table = torch.randperm(n_pages, generator=g)[:S * maxp].reshape(S, maxp).int()
    kc, vc = (torch.randn(n_pages, Hkv, page, D, generator=g).bfloat16() for _ in range(2))
    # distinct (sequence, slot) places; some tokens are padding
    place = torch.randperm(S * maxp * page, generator=g)[:tokens]
    seq, slot = (place // (maxp * page)).int(), (place % (maxp * page)).int()
    if tokens > 4:
        seq[::5] = -1 - seq[::5]
    posn = torch.randint(0, 100000, (tokens,), generator=g, dtype=torch.int32)
    qkv = torch.randn(tokens, Hq + 2 * Hkv, D, generator=g).bfloat16()
    qw = 1 + 0.3 * torch.randn(D, generator=g) if "q" in norm else None
    kw = 1 + 0.3 * torch.randn(D, generator=g) if "k" in norm else None
    freq = 10000.0 ** (-2 * torch.arange(rd // 2, dtype=torch.float64) / rd)
    x, dk, dv, dt, ds, dsl, dp, dqw, dkw, df = dev(qkv, kc, vc, table, seq, slot, posn, qw, kw, freq)
    parts = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if not strided:
        parts = [t.contiguous() for t in parts]
    out = torch.full((tokens, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got = bsa.cache_append(*parts, dk, dv, dt, ds, dsl, df, positions=dp if tokens != 5 else None, q_weight=dqw,
                           k_weight=dkw, interleaved=il, out=out)
    assert got is out and bsa.device_error() == 0
    p = posn.numpy() if tokens != 5 else slot.numpy()
    X = f64(qkv)
    yq, zq = ref_rows(X[:, :Hq], None if qw is None else f64(qw), p, freq.numpy(), 1e-6, 1.0, il)
    yk, zk = ref_rows(X[:, Hq:Hq + Hkv], None if kw is None else f64(kw), p, freq.numpy(), 1e-6, 1.0, il)
    on = (seq >= 0).numpy()
    within(f64(out)[on], zq[on], 2 * np.abs(yq[on]).max(-1, keepdims=True), "q")
    assert (f64(out)[~on] == 7).all()
    K, V = f64(kc), f64(vc)
    size = np.abs(K) * 0
    sq, sl = seq.numpy()[on], slot.numpy()[on]
    pg, r = table.numpy()[sq, sl // page], sl % page
    K[pg, :, r] = zk[on]
    size[pg, :, r] = 2 * np.abs(yk[on]).max(-1, keepdims=True)
    V[pg, :, r] = X[:, Hq + Hkv:][on]
    np.testing.assert_array_equal(f64(dv), V)
    gk = f64(dk)
    within(gk[pg, :, r], K[pg, :, r], size[pg, :, r], "k")
    gk[pg, :, r] = K[pg, :, r]
    np.testing.assert_array_equal(gk, K)  # nothing else was touched


@pytest.mark.parametrize("tokens,Hq,Hkv,D,page", [(7001, 10, 3, 64, 64), (5003, 1, 1, 128, 128), (2309, 33, 2, 128, 64)])
def test_append_of_many_tokens_is_that_of_few(bsa, tokens, Hq, Hkv, D, page):
    """Items in a row and token blocks that end inside a CTA, padding and bad places among
    them: the same rows bit for bit as from calls of a few tokens each."""
    g = torch.Generator().manual_seed(tokens)
    S, maxp = 40, -(-tokens // (40 * page)) + 2
    table = torch.randperm(S * maxp, generator=g).reshape(S, maxp).int()
    table[3, 1], table[5, 0] = -1, S * maxp
    place = torch.randperm(S * maxp * page, generator=g)[:tokens]
    seq, slot = (place // (maxp * page)).int(), (place % (maxp * page)).int()
    seq[torch.rand(tokens, generator=g) < 0.1] = -1
    seq[7], slot[11] = S, maxp * page
    w = (1 + 0.3 * torch.randn(D, generator=g)).cuda()
    x = torch.randn(tokens, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
    table, seq, slot = table.cuda(), seq.cuda(), slot.cuda()
    f = bsa.rope_inv_freq(D)
    got = []
    for step in (tokens, 7):
        kc, vc = (torch.zeros(S * maxp, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q = torch.zeros(tokens, Hq, D, dtype=torch.bfloat16, device="cuda")
        for i in range(0, tokens, step):
            y = x[i:i + step]
            bsa.cache_append(y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], kc, vc, table, seq[i:i + step],
                             slot[i:i + step], f, q_weight=w, out=q[i:i + step])
        assert bsa.device_error() == 32
        got.append((q, kc, vc))
    for s, t in zip(*got):
        assert torch.equal(s, t) and int((s != 0).sum()) > s.numel() // (8 if s is got[0][0] else 40)


def test_append_bad_places_are_reported_and_skipped(bsa):
    kc = torch.zeros(4, 2, 64, 64, device="cuda", dtype=torch.bfloat16)
    vc = torch.zeros_like(kc)
    table = torch.tensor([[0, 1, -1], [2, 99, -5]], dtype=torch.int32, device="cuda")
    x = torch.ones(8, 2, 64, device="cuda", dtype=torch.bfloat16)
    #       ok  id  slot<0  past  no page  bad page  bad page  ok
    seq = torch.tensor([0, 2, 0, 0, 0, 1, 1, 1], dtype=torch.int32, device="cuda")
    slot = torch.tensor([64, 0, -1, 192, 130, 64, 128, 5], dtype=torch.int32, device="cuda")
    bsa.cache_append(x, x, x, kc, vc, table, seq, slot)
    assert bsa.device_error() == 32
    want = torch.zeros_like(vc)
    want[1, :, 0] = 1
    want[2, :, 5] = 1
    assert torch.equal(vc, want) and torch.equal(kc, want)


@pytest.mark.parametrize("order", ["heads first", "batch last", "expanded", "reversed dims of one"])
def test_other_strides(bsa, order):
    """Views whose strides are not those of a fused projection."""
    B, N, H, D = 2, 37, 4, 64
    g = torch.Generator().manual_seed(3)
    x = torch.randn(B, N, H, D, generator=g).bfloat16().cuda()
    if order == "heads first":
        v = x.transpose(1, 2).contiguous().transpose(1, 2)
    elif order == "batch last":
        v = x.permute(1, 2, 0, 3).contiguous().permute(2, 0, 1, 3)
    elif order == "expanded":
        v = x[:, :, :1].expand(B, N, H, D)
    else:
        v = x[:1, :, :1].as_strided((1, N, 1, D), (5, H * D, 3, 1))
    f = bsa.rope_inv_freq(64)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")[None].expand(v.shape[0], N)
    w = torch.rand(D, device="cuda")
    args = dict(positions=pos, q_weight=w, k_weight=w)
    a = bsa.qk_norm_rope(v, v, v, f, **args)
    b = bsa.qk_norm_rope(v.contiguous(), v.contiguous(), v.contiguous(), f, **args)
    for s, t in zip(a, b):
        assert torch.equal(s, t)
    dz = [torch.randn_like(t) for t in a]
    ga = bsa.qk_norm_rope_backward(*dz, v, v, f, **args)
    gb = bsa.qk_norm_rope_backward(*dz, v.contiguous(), v.contiguous(), f, **args)
    for s, t in zip(ga, gb):
        assert torch.equal(s, t)


def test_gpu_refusals(bsa):
    """What only a CUDA tensor can get wrong: types, strides, shapes, streams, outputs."""
    x = torch.zeros(1, 8, 4, 64, device="cuda", dtype=torch.bfloat16)
    f, w = bsa.rope_inv_freq(64), torch.ones(64, device="cuda")
    bad = [dict(inv_freq=f.float()), dict(inv_freq=f[::2]), dict(positions=torch.arange(8, device="cuda")),
           dict(positions=torch.zeros(7, dtype=torch.int32, device="cuda")),
           dict(positions=torch.zeros(2, 8, dtype=torch.int32, device="cuda")),
           dict(positions=torch.zeros(8, dtype=torch.int32)), dict(q_weight=w[:32]), dict(q_weight=w.bfloat16()),
           dict(k_weight=w.cpu()), dict(q=x.float()), dict(q=x.transpose(2, 3)), dict(k=x[:, :4]),
           dict(k=x[..., :32]), dict(v=x[:, :, :2]), dict(out=(x, x, x)), dict(out=(x, x, None))]
    for kw in bad:
        with pytest.raises(ValueError):
            bsa.qk_norm_rope(**{**dict(q=x, k=x, v=x, inv_freq=f), **kw})
    for kw in (dict(kv_repeat=0), dict(eps=-1.0), dict(inv_freq=bsa.rope_inv_freq(24)),
               dict(inv_freq=bsa.rope_inv_freq(80)), dict(q=torch.zeros(1, 8, 4, 68, device="cuda",
                                                                       dtype=torch.bfloat16)[..., :64]),
               dict(q=torch.zeros(2056, device="cuda", dtype=torch.bfloat16)[1:2049].view(1, 8, 4, 64))):
        with pytest.raises(bsa.BsaError):
            bsa.qk_norm_rope(**{**dict(q=x, k=x, v=x, inv_freq=f), **kw})
    z = torch.zeros(1, 4, 8, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bsa.qk_norm_rope_backward(z.transpose(1, 2), z, z, x, x, f)
    with pytest.raises(bsa.BsaError):  # gradient rows that coincide
        bsa.qk_norm_rope_backward(z, z, z, x, x, f, out=(x, x, x[:, :, :1].expand(1, 8, 4, 64)))
    assert bsa.device_error() == 0


def test_far_rows(bsa):
    """Token rows and pages whose offsets pass 2^31 bytes and 2^31 elements."""
    n = 2 ** 31 // 128 + 3000  # rows of 128 values
    pool = torch.empty(n, 128, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(40, 128, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    pool[-40:] = x
    far = pool[-40:].view(1, 40, 1, 128)
    near = x.view(1, 40, 1, 128)
    f = bsa.rope_inv_freq(128)
    assert far.storage_offset() > 2 ** 31
    step = pool.as_strided((1, 2, 1, 128), (0, (n - 1) * 128, 0, 1))  # two tokens, the second one far
    pool[0] = x[3]
    for a, b in ((far, near), (step, torch.stack([x[3], x[-1]]).view(1, 2, 1, 128))):
        za, zb = bsa.qk_norm_rope(a, a, a, f), bsa.qk_norm_rope(b, b, b, f)
        assert all(torch.equal(s, t) for s, t in zip(za, zb))
    # a cache of the same size: its last page
    pages = n // 64
    cache = pool[:pages * 64].view(pages, 1, 64, 128)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.cache_append(near[0, :1], near[0, :1], near[0, :1], cache, cache, table, one, one + 63, None)
    assert torch.equal(cache[pages - 1, 0, 63], x[0]) and bsa.device_error() == 0
