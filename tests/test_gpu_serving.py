"""The calls in a row, as a model uses them: a projection through the
block-sparse attention and its gradients; a prompt, drafted trees, acceptance,
forks and defragmentation over one cache; and a decoding step captured into a
graph that replays while the lengths advance on the device."""

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


def norm_rope64(x, w, pos, freq):
    """[tokens, H, D] float64, halves layout."""
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    ang = pos.double()[:, None] * freq
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    h = freq.numel()
    a, b = y[..., :h], y[..., h:2 * h]
    return torch.cat([a * c - b * s, b * c + a * s, y[..., 2 * h:]], -1)


def test_projection_to_gradients(bsa):
    """qk_norm_rope -> forward -> backward -> qk_norm_rope_backward against
    autograd in 64 bits.  Bound: the attention's gradients are held to 2e-2 of
    their largest value (2e-3 in the mean) for exact inputs; q and k arrive
    rounded to bf16, which acts on the scores like the rounding of P that this
    covers, and the rest is linear with fp32 arithmetic and one more rounding:
    twice that."""
    N, Hq, Hkv, D, block = 512, 4, 2, 64, 64
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(1, N, Hq + 2 * Hkv, D, generator=g).bfloat16()
    qw, kw = 1 + 0.2 * torch.randn(D, generator=g), 1 + 0.2 * torch.randn(D, generator=g)
    do = torch.randn(1, Hq, N, D, generator=g).bfloat16()
    freq = bsa.rope_inv_freq(D)
    x = qkv.cuda()
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    args = dict(q_weight=qw.cuda(), k_weight=kw.cuda(), kv_repeat=Hq // Hkv)
    Q, K, V = bsa.qk_norm_rope(q, k, v, freq, **args)
    pat = bsa.Pattern(N // block, 2, 0, True, (0,))
    rp, ci = bsa.build_mask_csr(pat, 1, Hq)
    O, lse = bsa.forward(Q, K, V, rp, ci, block, causal=True)
    dQ, dK, dV = bsa.backward(Q, K, V, O, do.cuda(), lse, rp, ci, block, causal=True)
    dx = torch.empty_like(x)
    out = (dx[:, :, :Hq], dx[:, :, Hq:Hq + Hkv], dx[:, :, Hq + Hkv:])
    *_, dqw, dkw = bsa.qk_norm_rope_backward(dQ, dK, dV, q, k, freq, out=out, **args)
    assert bsa.device_error() == 0
    # 64 bits
    X, QW, KW = qkv[0].double().requires_grad_(), qw.double().requires_grad_(), kw.double().requires_grad_()
    pos, fr = torch.arange(N), freq.cpu()
    zq = norm_rope64(X[:, :Hq], QW, pos, fr).transpose(0, 1)
    zk = norm_rope64(X[:, Hq:Hq + Hkv], KW, pos, fr).transpose(0, 1).repeat_interleave(Hq // Hkv, 0)
    zv = X[:, Hq + Hkv:].transpose(0, 1).repeat_interleave(Hq // Hkv, 0)
    bi = torch.arange(N) // block
    see = ((bi[:, None] - bi[None] <= 2) | (bi[None] == 0)) & (torch.arange(N)[:, None] >= torch.arange(N)[None])
    S = (zq @ zk.transpose(1, 2) / D ** 0.5).masked_fill(~see, -float("inf"))
    ((torch.softmax(S, -1) @ zv) * do[0].double()).sum().backward()
    for got, ref, what in ((dx[0], X.grad, "projection"), (dqw, QW.grad, "q weight"), (dkw, KW.grad, "k weight")):
        d, G = (got.detach().cpu().double() - ref).abs(), ref.abs().max()
        assert d.max() <= 4e-2 * G and d.mean() <= 4e-3 * G, (what, float(d.max() / G), float(d.mean() / G))


def attend64(q, K, V, see, scale):
    """q [T,G,D], K, V [S,D], see [T,S]: O and LSE."""
    S = torch.einsum("tgd,sd->tgs", q, K) * scale
    S = S.masked_fill(~see[:, None], -float("inf"))
    return torch.softmax(S, -1) @ V, torch.logsumexp(S, -1)


def test_serving_steps(bsa):
    """Two prompts in one cache, drafted trees, acceptance, a fork that goes on
    by itself, a defragmentation; after every step the attention of the newest
    tokens against 64 bits over rows kept outside the cache (the bf16 rows that
    the calls wrote; P in two bf16 parts, one rounding of the result:
    |O| 2^-8 + 2^-12 of the weighted |v|, the derivation of test_gpu_tree.py
    without its rounding of P, at scores below 30)."""
    Hq, Hkv, D, page, S, P = 8, 2, 128, 64, 4, 12
    G, scale, freq = Hq // Hkv, D ** -0.5, bsa.rope_inv_freq(128, 500000.0, "linear", 2.0)
    g = torch.Generator().manual_seed(5)
    kc, vc = (torch.full((40, Hkv, page, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.full((S, P), -1, dtype=torch.int32, device="cuda")
    ref = torch.zeros(40, dtype=torch.int32, device="cuda")
    qw, kw = torch.rand(D, device="cuda") + 0.5, torch.rand(D, device="cuda") + 0.5
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    history = {}  # sequence -> (K rows, V rows), float64 [Hkv, n, D]

    def project(n):
        x = torch.randn(n, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]

    def rows(seq, slots):
        s = torch.tensor(slots)
        pg = table[seq].cpu()[s // page].long()
        return [t.cpu().double()[pg, :, s % page].transpose(0, 1) for t in (kc, vc)]

    def append(seq, slots, pos, parts):
        sid = torch.full((len(slots),), seq, dtype=torch.int32, device="cuda")
        return bsa.cache_append(*parts, kc, vc, table, sid, i32(*slots), freq, positions=i32(*pos), q_weight=qw,
                                k_weight=kw)

    def check(seq_of, q, o, lse, see_of):
        for r, s in enumerate(seq_of):
            K, V = history[s]
            for h in range(Hkv):
                O, L = attend64(q[r, :, h * G:(h + 1) * G].cpu().double(), K[h], V[h], see_of[r], scale)
                A = attend64(q[r, :, h * G:(h + 1) * G].cpu().double(), K[h], V[h].abs(), see_of[r], scale)[0]
                n = see_of[r].shape[0]
                d = (o[r, :n, h * G:(h + 1) * G].cpu().double() - O).abs()
                assert (d <= O.abs() * 2.0 ** -8 + A * 2.0 ** -12).all()
                assert (lse[r, :n, h * G:(h + 1) * G].cpu().double() - L).abs().max() <= 2.0 ** -12

    # prompts of 130 and 64 tokens; the same rows as the training path gives
    lens = {0: 130, 1: 64}
    assert bsa.cache_resize(table, ref, i32(0, 1), i32(0, 0), i32(130 + 8, 64 + 8), kc, vc).tolist() == [1, 1]
    for s, n in lens.items():
        parts = project(n)
        q = append(s, range(n), range(n), parts)
        Q, K, V = bsa.qk_norm_rope(*(t[None] for t in parts), freq, q_weight=qw, k_weight=kw)
        assert torch.equal(q.transpose(0, 1), Q[0])
        history[s] = rows(s, range(n))
        assert torch.equal(history[s][0], K[0].cpu().double()) and torch.equal(history[s][1], V[0].cpu().double())
    # a tree of five drafts each: 0 - 1 - 3, 0 - 2 - 4
    T, depth, up = 5, [0, 1, 1, 2, 2], [None, 0, 0, 1, 2]
    bits = []
    for u in range(T):
        bits.append((bits[up[u]] if up[u] is not None else 0) | 1 << u)
    see_tree = torch.tensor([[bool(b >> u & 1) for u in range(T)] for b in bits])
    mask = torch.tensor([bits, bits], dtype=torch.int64, device="cuda")
    q = []
    for s in (0, 1):
        n = lens[s]
        q.append(append(s, range(n, n + T), [n + d for d in depth], project(T)))
    q = torch.stack(q)
    ctx = i32(lens[0], lens[1])
    o, lse = bsa.tree_attention(q, kc, vc, table[:2], ctx, tree_mask=mask)
    kept = {s: history[s] for s in (0, 1)}
    for s in (0, 1):
        history[s] = [torch.cat([a, b], 1) for a, b in zip(kept[s], rows(s, range(lens[s], lens[s] + T)))]
    check((0, 1), q, o, lse, [torch.cat([torch.ones(T, lens[s], dtype=torch.bool), see_tree], 1) for s in (0, 1)])
    # sequence 0 accepts 0 - 2 - 4, sequence 1 only 0
    new = bsa.cache_accept(kc, vc, table[:2], ctx, i32(0, 2, 4, 0, 0, 0, 0, 0, 0, 0).reshape(2, 5), i32(3, 1))
    assert new.tolist() == [133, 65]
    for s, acc in ((0, [0, 2, 4]), (1, [0])):
        history[s] = [torch.cat([a[:, :lens[s]], a[:, [lens[s] + u for u in acc]]], 1) for a in history[s]]
        lens[s] = int(new[s])
        k, v = rows(s, range(lens[s]))
        assert torch.equal(k, history[s][0]) and torch.equal(v, history[s][1])
    # beams: 2 and 3 fork from 0 and go on with tokens of their own; 1 is freed
    assert bsa.cache_fork(table, ref, i32(0, 0), i32(2, 3), i32(133, 133), kc, vc).tolist() == [1, 1]
    ones = bsa.cache_resize(table, ref, i32(1, 0, 2, 3), i32(0, 133, 133, 133), i32(0, 200, 200, 200), kc, vc)
    assert ones.tolist() == [1, 1, 1, 1]
    for s in (0, 2, 3):
        q = append(s, [133], [133], project(1))
        history[s] = [torch.cat([a[:, :133], b], 1) for a, b in zip(history[0], rows(s, [133]))]
        o, lse = bsa.tree_attention(q[None], kc, vc, table[s:s + 1], i32(133))
        check((s,), q[None], o, lse, [torch.ones(1, 134, dtype=torch.bool)])
    # defragmentation changes places, not results; and lists of pages name what they did before
    q = project(3)[0][:, None].contiguous()
    seqs = torch.tensor([0, 2, 3])
    lists = (i32(0, 2, 3, 5, 6, 8, 9), i32(0, 2, 1, 2, 0, 1, 0, 2, 1))
    # (rows: sequence, key head; the newest token is at slot 133, page 2)
    before = [bsa.tree_attention(q, kc, vc, table[seqs.cuda()], i32(133, 133, 133)),
              bsa.tree_attention(q, kc, vc, table[seqs.cuda()], i32(133, 133, 133), row_ptr=lists[0],
                                 col_idx=lists[1])]
    old = ref.clone()
    bsa.cache_compact(table, ref, kc, vc)
    live = int((old > 0).sum())
    assert (ref[:live] > 0).all() and (ref[live:] == 0).all()
    after = [bsa.tree_attention(q, kc, vc, table[seqs.cuda()], i32(133, 133, 133)),
             bsa.tree_attention(q, kc, vc, table[seqs.cuda()], i32(133, 133, 133), row_ptr=lists[0],
                                col_idx=lists[1])]
    for x, y in zip(before, after):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    assert bsa.device_error() == 0


def test_decoding_step_in_a_graph(bsa):
    """append + attention + accept captured once; replays see the lengths, slots
    and inputs that the device holds then, and match eager calls bit for bit."""
    B, Hq, Hkv, D, page = 3, 8, 2, 64, 128
    g = torch.Generator().manual_seed(9)
    start = [5, 126, 300]
    table = torch.arange(B * 4, dtype=torch.int32).reshape(B, 4).cuda()
    pools = [torch.randn(B * 4, Hkv, page, D, generator=g).bfloat16().cuda() for _ in range(2)]
    freq = bsa.rope_inv_freq(64)
    x = torch.zeros(B, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    seq = torch.arange(B, dtype=torch.int32, device="cuda")
    zero, one = torch.zeros(B, 1, dtype=torch.int32, device="cuda"), torch.ones(B, dtype=torch.int32, device="cuda")

    def step(kc, vc, ctx):
        q = bsa.cache_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kc, vc, table, seq, ctx, freq)
        o, _ = bsa.tree_attention(q[:, None], kc, vc, table, ctx)
        ctx.copy_(bsa.cache_accept(kc, vc, table, ctx, zero, one))
        return o

    eager, graphed = [[t.clone() for t in pools] + [torch.tensor(start, dtype=torch.int32).cuda()] for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*graphed)
    graphed[2].copy_(torch.tensor(start, dtype=torch.int32))
    for t, p in zip(graphed, pools):
        t.copy_(p)
    for i in range(6):
        x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        graph.replay()
        want = step(*eager)
        assert torch.equal(out, want), i
    assert graphed[2].tolist() == [s + 6 for s in start] == eager[2].tolist()
    assert torch.equal(graphed[0], eager[0]) and torch.equal(graphed[1], eager[1]) and bsa.device_error() == 0


def test_calls_keep_nothing(bsa):
    """Memory and reference counts are what they were after many calls, refused ones among them."""
    import sys
    x = torch.randn(1, 16, 6, 64, device="cuda").bfloat16()
    q, k, v = x[:, :, :2], x[:, :, 2:4], x[:, :, 4:]
    f, w = bsa.rope_inv_freq(64), torch.ones(64, device="cuda")
    kc, vc = (torch.zeros(4, 2, 64, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table = torch.arange(4, dtype=torch.int32, device="cuda").reshape(2, 2)
    ref = torch.ones(4, dtype=torch.int32, device="cuda")
    two, one = torch.tensor([70, 3], dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    out = torch.empty(2, 1, 4, 64, device="cuda", dtype=torch.bfloat16)
    q1 = torch.randn(2, 1, 4, 64, device="cuda").bfloat16()

    def everything():
        z = bsa.qk_norm_rope(q, k, v, f, q_weight=w)
        bsa.qk_norm_rope_backward(*z, q, k, f, q_weight=w)
        bsa.cache_append(k[0], k[0], v[0], kc, vc, table, two.repeat(8) * 0, two.repeat(8) * 0, f)
        assert bsa.tree_attention(q1, kc, vc, table, two, out=out)[0] is out
        bsa.tree_attention(q1, kc, vc, table, two)
        bsa.cache_accept(kc, vc, table, two, one.reshape(2, 1) * 0, one)
        bsa.cache_resize(table, ref, one * 0, two, two, kc, vc)
        bsa.cache_compact(table, ref, kc, vc)
        for bad in (lambda: bsa.qk_norm_rope(q, k, v, [1.0]), lambda: bsa.qk_norm_rope(q, k, v, f, eps=-1.0),
                    lambda: bsa.tree_attention(q1, kc, vc, table, None), lambda: bsa.cache_compact(table, ref, kc, out)):
            with pytest.raises((ValueError, bsa.BsaError)):
                bad()
        with pytest.raises(TypeError):
            bsa.qk_norm_rope(q, k, v, f, kv_repeat=1.5)

    held = (x, q, k, v, f, w, kc, vc, table, ref, two, one, out, q1)
    everything()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated(), [sys.getrefcount(t) for t in held]
    for _ in range(50):
        everything()
    torch.cuda.synchronize()
    assert (torch.cuda.memory_allocated(), [sys.getrefcount(t) for t in held]) == before
    bsa.device_error()


def test_calls_from_two_threads(bsa):
    """Calls at once from two threads, each on its own stream, with results of their own."""
    import threading
    f = bsa.rope_inv_freq(128)
    g = torch.Generator().manual_seed(2)
    data = [torch.randn(1, 300 + 100 * i, 12, 128, generator=g).bfloat16().cuda() for i in range(2)]

    def step(x):
        return bsa.qk_norm_rope(x[:, :, :8], x[:, :, 8:10], x[:, :, 10:], f, kv_repeat=4)

    want = [[t.clone() for t in step(x)] for x in data]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(200):
                got = step(data[i])
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and bsa.device_error() == 0
