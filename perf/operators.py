"""Cases, plain forms and 64-bit references of the operators around block-sparse attention.

Four families:

* ``norm_rope``: the RMS norm of every query and key head with the position rotation in
  the same pass, from token-major projections to the head-major tensors that the
  attention takes, and (``grad``) its gradients;
* ``append``: the same for the new tokens of a served batch, keys and values going into
  the pages of a cache; with more than one drafted token per sequence, followed by the
  compaction of the accepted ones;
* ``tree``: attention of the drafted tokens of each sequence (one or a tree) over its
  pages, over all of them or over a block list per key head;
* ``pages``: sequences that take over another's pages (``fork``), and live pages moved to
  the front of the pool (``compact``).

``own`` False: elementary torch operations in 32 bits (64 for angles and for the sums over
all tokens).  ``own`` True: the calls of the package.
"""

from __future__ import annotations

import math
import random

import torch

own = False


def _bsa():
    import block_sparse_flashattention_bsa_gb300 as bsa
    return bsa


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest sequence of the attention's own configurations: the launch counts
        dict(name="prep_1k", op="norm_rope", grad=False, B=1, N=1024, Hq=2, Hkv=2, rep=1, D=64, rd=64,
             interleaved=False, norm=True, factor=1.0, packed=False),
        # a 128K prompt, grouped key heads repeated for an attention with one key head per query head
        dict(name="prep_128k", op="norm_rope", grad=False, B=1, N=131072, Hq=32, Hkv=8, rep=4, D=128, rd=128,
             interleaved=False, norm=True, factor=8.0, packed=False),
        # training at 16K: the gradients on their way from the attention to the projection
        dict(name="grad_16k", op="norm_rope", grad=True, B=1, N=16384, Hq=16, Hkv=16, rep=1, D=128, rd=128,
             interleaved=False, norm=True, factor=1.0, packed=False),
        # packed documents of odd lengths, part of the head rotated, pairs interleaved
        dict(name="grad_packed", op="norm_rope", grad=True, B=2, N=4099, Hq=20, Hkv=5, rep=4, D=64, rd=32,
             interleaved=True, norm=True, factor=1.0, packed=True),
        # one token of one stream
        dict(name="append_one", op="append", B=1, T=1, Hq=16, Hkv=16, D=128, rd=128, page=128, ctx=3000,
             interleaved=False, norm=True),
        # a verification step of a large batch: eight drafted tokens a sequence, then the accepted ones move up
        dict(name="append_drafts", op="append", B=256, T=8, Hq=32, Hkv=8, D=128, rd=64, page=128, ctx=900,
             interleaved=True, norm=False),
        # one stream, short context: latency
        dict(name="decode_one", op="tree", B=1, T=1, Hq=16, Hkv=2, D=64, page=64, ctx=1500, ragged=False,
             listed_pages=0),
        # a served batch of ragged contexts, one token each
        dict(name="decode_batch", op="tree", B=96, T=1, Hq=32, Hkv=8, D=128, page=128, ctx=8192, ragged=True,
             listed_pages=0),
        # trees of drafted tokens over 128K contexts
        dict(name="tree_128k", op="tree", B=4, T=16, Hq=32, Hkv=8, D=128, page=128, ctx=131000, ragged=False,
             listed_pages=0),
        # block lists: sink, window and selected pages of long contexts, short drafts
        dict(name="tree_listed", op="tree", B=32, T=5, Hq=16, Hkv=16, D=128, page=64, ctx=32768, ragged=True,
             listed_pages=24),
        # a beam step over every layer: the lost beams' pages go back, the kept ones are forked
        dict(name="fork_beams", op="pages", call="fork", n=64, layers=8, Hkv=8, D=128, page=128, pages=3000,
             ctx=2000),
        # defragmentation of a pool that is 60 % live
        dict(name="compact_pool", op="pages", call="compact", n=48, layers=2, Hkv=8, D=128, page=64, pages=4096,
             ctx=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["norm_rope", "norm_rope", "append", "tree", "tree", "tree", "pages"])
    D = rng.choice([64, 128])
    if op == "norm_rope":
        Hkv = _log(rng, 1, 16)
        G = rng.choice([1, 1, 2, 3, 4, 8])
        Hq = min(48, Hkv * G)
        G = Hq // Hkv
        Hq = Hkv * G
        rep = rng.choice([1, G])
        B = rng.choice([1, 1, 2, 3])
        most = 131072 * 96 * 128 // ((Hq + 2 * Hkv * rep) * D * B * 2)
        return dict(op=op, grad=rng.random() < 0.5, B=B, N=_log(rng, 64, min(131072, most)), Hq=Hq, Hkv=Hkv, rep=rep,
                    D=D, rd=rng.choice([16, 32, D // 2, D, D]), interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.8, factor=rng.choice([1.0, 1.0, 4.0, 16.0]), packed=rng.random() < 0.3)
    Hkv = rng.choice([1, 2, 3, 4, 8, 8, 16])
    page = rng.choice([64, 128])
    if op == "append":
        return dict(op=op, B=_log(rng, 1, 256), T=rng.choice([1, 1, 2, 4, 7, 16]), Hq=Hkv * rng.choice([1, 2, 4, 5]),
                    Hkv=Hkv, D=D, rd=rng.choice([16, D // 2, D, D]), page=page, ctx=_log(rng, 1, 2000),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.7)
    if op == "tree":
        T = rng.choice([1, 1, 2, 4, 8, 13, 32, 64])
        G = rng.choice([1, 2, 4, 5, 8])
        ctx = _log(rng, 1, 131072)
        most = 131000 * 4 * 8 * 128 * 64 // (ctx * Hkv * D * max(64, T * G))
        B = _log(rng, 1, max(1, min(128, most)))
        return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, ctx=ctx, ragged=rng.random() < 0.6,
                    listed_pages=rng.choice([0, 0, 8, 19, 32]))
    pages = _log(rng, 200, 3000)
    layers = rng.choice([1, 2, 3, 4])
    return dict(op=op, call=rng.choice(["fork", "compact"]), n=_log(rng, 2, 48), layers=layers,
                Hkv=rng.choice([1, 2, 4, 8]), D=D, page=page, pages=pages, ctx=_log(rng, 10, 1500))


# ------------------------------------------------------------------ inputs
def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFF)
    return g


def _randn(shape, g, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32 if dtype == torch.float32 else dtype)
            * scale).to(dtype)


def _inv_freq(rd, factor):
    """base 10000; a factor above 1 stretches the slow rotations (a ramp between 1 and 32
    turns over 8192 positions), as checkpoints extended to long contexts have it."""
    i = torch.arange(rd // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rd)
    if factor > 1.0:
        ramp = ((8192.0 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
        f = f * (ramp + (1 - ramp) / factor)
    return f.cuda()


def _weights(norm, D, g):
    if not norm:
        return None, None
    return (1 + 0.2 * _randn((D,), g, torch.float32)), (1 + 0.2 * _randn((D,), g, torch.float32))


def prepare(case, seed):
    return {"norm_rope": _prepare_norm_rope, "append": _prepare_append, "tree": _prepare_tree,
            "pages": _prepare_pages}[case["op"]](case, seed)


def _prepare_norm_rope(c, seed):
    g, r = _gen(seed), random.Random(seed)
    B, N, Hq, Hkv, D = c["B"], c["N"], c["Hq"], c["Hkv"], c["D"]
    s = dict(c)
    # one fused projection; q, k and v are views of it, as a model's split gives them
    s["qkv"] = _randn((B, N, Hq + 2 * Hkv, D), g)
    s["inv_freq"] = _inv_freq(c["rd"], c["factor"])
    s["gain"] = 1.0 if c["factor"] == 1.0 else 0.1 * math.log(c["factor"]) + 1.0
    s["qw"], s["kw"] = _weights(c["norm"], D, g)
    s["pos"] = None
    if c["packed"]:
        rows = []
        for _ in range(B):
            p = []
            while len(p) < N:
                p += range(r.randint(1, max(2, N // 2)))
            rows.append(torch.tensor(p[:N], dtype=torch.int32))
        s["pos"] = torch.stack(rows).cuda()
    if c["grad"]:
        H2 = Hkv * c["rep"]
        s["dz"] = tuple(_randn((B, H, N, D), g) for H in (Hq, H2, H2))
    return s


def _table(lens, most, page, extra, r):
    """A page table of sequences that hold `lens` slots of at most `most`, physical pages in
    random order from a pool that would hold them all at that length."""
    held = [-(-n // page) for n in lens]
    P = -(-most // page)
    order = list(range(P * len(lens) + extra))
    r.shuffle(order)
    t, at = torch.full((len(lens), P), -1, dtype=torch.int32), 0
    for i, h in enumerate(held):
        t[i, :h] = torch.tensor(order[at:at + h], dtype=torch.int32)
        at += h
    return t, len(order)


def _prepare_append(c, seed):
    g, r = _gen(seed), random.Random(seed)
    B, T, Hq, Hkv, D, page = (c[x] for x in ("B", "T", "Hq", "Hkv", "D", "page"))
    s = dict(c)
    ctx = [r.randint(max(0, c["ctx"] // 2), c["ctx"]) for _ in range(B)]
    t, n = _table([x + T for x in ctx], c["ctx"] + T, page, 3, r)
    s["table"] = t.cuda()
    s["kc"], s["vc"] = (_randn((n, Hkv, page, D), g) for _ in range(2))
    s["qkv"] = _randn((B * T, Hq + 2 * Hkv, D), g)
    s["inv_freq"], (s["qw"], s["kw"]) = _inv_freq(c["rd"], 1.0), _weights(c["norm"], D, g)
    depth = [0] * T
    for u in range(1, T):  # a tree: each draft hangs under an earlier one
        depth[u] = depth[r.randrange(u)] + 1
    cx = torch.tensor(ctx, dtype=torch.int32)
    s["ctx"] = cx.cuda()
    s["seq"] = torch.arange(B, dtype=torch.int32).repeat_interleave(T).cuda()
    s["slot"] = (cx[:, None] + torch.arange(T, dtype=torch.int32)[None]).reshape(-1).contiguous().cuda()
    s["pos"] = (cx[:, None] + torch.tensor(depth, dtype=torch.int32)[None]).reshape(-1).contiguous().cuda()
    acc, na = torch.zeros((B, T), dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        k = r.randint(1, T)
        acc[b, :k] = torch.tensor(sorted(r.sample(range(T), k)), dtype=torch.int32)
        na[b] = k
    s["acc"], s["na"] = acc.cuda(), na.cuda()
    return s


def _prepare_tree(c, seed):
    g, r = _gen(seed), random.Random(seed)
    B, T, Hq, Hkv, D, page = (c[x] for x in ("B", "T", "Hq", "Hkv", "D", "page"))
    s = dict(c)
    ctx = [r.randint(max(0, c["ctx"] // 8), c["ctx"]) if c["ragged"] else c["ctx"] for _ in range(B)]
    t, n = _table([x + T for x in ctx], c["ctx"] + T, page, 2, r)
    s["table"] = t.cuda()
    s["kc"], s["vc"] = (_randn((n, Hkv, page, D), g) for _ in range(2))
    s["q"] = _randn((B, T, Hq, D), g, scale=1.5)
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32).cuda()
    s["dl"], s["mask"] = None, None
    if T > 1:
        dl = [r.randint(max(1, T // 2), T) if c["ragged"] else T for _ in range(B)]
        m = torch.zeros((B, T), dtype=torch.int64)
        for b in range(B):
            bits = []
            for u in range(T):
                w = (bits[r.randrange(u)] if u else 0) | (1 << u)
                bits.append(w)
                m[b, u] = w if w < 1 << 63 else w - (1 << 64)
        s["dl"], s["mask"] = torch.tensor(dl, dtype=torch.int32).cuda(), m.cuda()
        # rows behind a sequence's drafts are no outputs: both sides start from zeros
    s["o"] = torch.zeros((B, T, Hq, D), device="cuda", dtype=torch.bfloat16)
    s["lse"] = torch.zeros((B, T, Hq), device="cuda", dtype=torch.float32)
    s["rp"], s["ci"] = None, None
    if c["listed_pages"]:
        rp, ci = [0], []
        for b in range(B):
            held = -(-(ctx[b] + T) // page)
            for _ in range(Hkv):
                last = list(range(max(0, held - 4), held))
                rest = [j for j in r.sample(range(held), min(held, c["listed_pages"])) if j not in last and j]
                row = sorted({0, *last, *rest[:max(0, c["listed_pages"] - 5)]})
                ci += row
                rp.append(len(ci))
        s["rp"], s["ci"] = torch.tensor(rp, dtype=torch.int32).cuda(), torch.tensor(ci, dtype=torch.int32).cuda()
    return s


def _prepare_pages(c, seed):
    g, r = _gen(seed), random.Random(seed)
    n, L, Hkv, D, page, pages = (c[x] for x in ("n", "layers", "Hkv", "D", "page", "pages"))
    s = dict(c)
    s["kc"], s["vc"] = (_randn((L, pages, Hkv, page, D), g) for _ in range(2))
    ref = torch.zeros(pages, dtype=torch.int32)
    order = list(range(pages))
    r.shuffle(order)
    if c["call"] == "fork":
        # n sequences, half of them beams to be replaced by forks of the other half
        half = max(1, n // 2)
        most = max(1, (pages - n) // half) * page
        lens = [min(most, r.randint(max(1, c["ctx"] // 2), c["ctx"])) for _ in range(half)]
        P = -(-min(most, c["ctx"]) // page)
        t, at = torch.full((2 * half, P), -1, dtype=torch.int32), 0
        for i, x in enumerate(lens):
            h = -(-x // page)
            t[i, :h] = torch.tensor(order[at:at + h], dtype=torch.int32)
            at += h
        src = [r.randrange(half) for _ in range(half)]
        s["src"] = torch.tensor(src, dtype=torch.int32).cuda()
        s["dst"] = torch.arange(half, 2 * half, dtype=torch.int32).cuda()
        s["lens"] = torch.tensor([lens[i] for i in src], dtype=torch.int32).cuda()
        s["zero"] = torch.zeros(half, dtype=torch.int32).cuda()
    else:
        # n sequences over 60 % of the pool, some pages shared by two of them
        live = max(1, int(0.6 * pages))
        P = -(-live // n) + 3
        t, at = torch.full((n, P), -1, dtype=torch.int32), 0
        for i in range(n):
            h = min(P - 3, live - at)
            row = order[at:at + h]
            if i and at:
                row = [order[r.randrange(at)] for _ in range(2)] + row
            t[i, :len(row)] = torch.tensor(row, dtype=torch.int32)
            at += h
    for x in t[t >= 0].tolist():
        ref[x] += 1
    s["table"], s["ref"] = t.cuda(), ref.cuda()
    s["table0"], s["ref0"] = s["table"].clone(), s["ref"].clone()
    return s


# ------------------------------------------------------------------ run
def run(state):
    return {"norm_rope": _run_norm_rope, "append": _run_append, "tree": _run_tree,
            "pages": _run_pages}[state["op"]](state)


def _split(x, Hq, Hkv):
    return x[..., :Hq, :], x[..., Hq:Hq + Hkv, :], x[..., Hq + Hkv:, :]


def _angles(pos, inv_freq, gain):
    a = pos.to(torch.float64)[..., None] * inv_freq
    return (a.cos() * gain).float(), (a.sin() * gain).float()  # [..., rd/2]


def _pairs(y, rd, interleaved):
    if interleaved:
        return y[..., 0:rd:2], y[..., 1:rd:2]
    return y[..., :rd // 2], y[..., rd // 2:rd]


def _rotated(y, cos, sin, rd, interleaved):
    """y [..., H, D] in 32 bits; cos, sin [..., rd/2] of the token."""
    a, b = _pairs(y, rd, interleaved)
    c, s = cos[..., None, :], sin[..., None, :]
    out = y.clone()
    oa, ob = _pairs(out, rd, interleaved)
    ta, tb = a * c - b * s, b * c + a * s
    oa.copy_(ta)
    ob.copy_(tb)
    return out


def _normed(x, w, eps=1e-6):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w


def _positions(s, B, N):
    return s["pos"] if s["pos"] is not None else torch.arange(N, device="cuda", dtype=torch.int32)[None].expand(B, N)


def _run_norm_rope(s):
    Hq, Hkv, rd, il, rep = s["Hq"], s["Hkv"], s["rd"], s["interleaved"], s["rep"]
    q, k, v = _split(s["qkv"], Hq, Hkv)
    if own:
        bsa = _bsa()
        more = dict(positions=s["pos"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, gain=s["gain"],
                    interleaved=il, kv_repeat=rep)
        if not s["grad"]:
            return bsa.qk_norm_rope(q, k, v, s["inv_freq"], **more)
        return bsa.qk_norm_rope_backward(*s["dz"], q, k, s["inv_freq"], **more)
    B, N = q.shape[:2]
    cos, sin = _angles(_positions(s, B, N), s["inv_freq"], s["gain"])
    if not s["grad"]:
        zq = _rotated(_normed(q, s["qw"]), cos, sin, rd, il).to(torch.bfloat16)
        zk = _rotated(_normed(k, s["kw"]), cos, sin, rd, il).to(torch.bfloat16)
        zk, zv = (x.transpose(1, 2).repeat_interleave(rep, dim=1) for x in (zk, v))
        return zq.transpose(1, 2).contiguous(), zk.contiguous(), zv.contiguous()
    dq, dk, dv = s["dz"]
    out = []
    for x, w, dz, r in ((q, s["qw"], dq, 1), (k, s["kw"], dk, rep)):
        d = dz.float().transpose(1, 2)  # [B, N, H * r, D]
        d = d.reshape(B, N, x.shape[2], r, d.shape[-1]).sum(3)
        dy = _rotated(d, cos, -sin, rd, il)
        if w is None:
            out.append((dy.to(torch.bfloat16), None))
            continue
        x = x.float()
        rr = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        xh, g = x * rr, dy * w
        dx = rr * (g - xh * (g * xh).mean(-1, keepdim=True))
        out.append((dx.to(torch.bfloat16), (dy * xh).sum((0, 1, 2), dtype=torch.float64).float()))
    D = dv.shape[-1]
    gv = dv.float().transpose(1, 2).reshape(B, N, Hkv, rep, D).sum(3).to(torch.bfloat16)
    return out[0][0], out[1][0], gv, out[0][1], out[1][1]


def _run_append(s):
    Hq, Hkv, T, rd, il, page = s["Hq"], s["Hkv"], s["T"], s["rd"], s["interleaved"], s["page"]
    q, k, v = _split(s["qkv"], Hq, Hkv)
    if own:
        bsa = _bsa()
        zq = bsa.cache_append(q, k, v, s["kc"], s["vc"], s["table"], s["seq"], s["slot"], s["inv_freq"],
                              positions=s["pos"], q_weight=s["qw"], k_weight=s["kw"], interleaved=il)
        if T == 1:
            return zq, s["kc"], s["vc"]
        new = bsa.cache_accept(s["kc"], s["vc"], s["table"], s["ctx"], s["acc"], s["na"])
        return zq, s["kc"], s["vc"], new
    cos, sin = _angles(s["pos"], s["inv_freq"], 1.0)
    zq = _rotated(_normed(q, s["qw"]), cos, sin, rd, il).to(torch.bfloat16)
    zk = _rotated(_normed(k, s["kw"]), cos, sin, rd, il).to(torch.bfloat16)
    pg = s["table"][s["seq"].long(), (s["slot"] // page).long()].long()
    at = (s["slot"] % page).long()
    s["kc"][pg, :, at] = zk
    s["vc"][pg, :, at] = v
    if T == 1:
        return zq, s["kc"], s["vc"]
    # accepted rows: where a draft stays out, the row is written back to itself
    B = s["ctx"].shape[0]
    i = torch.arange(T, device="cuda")[None].expand(B, T)
    take = torch.where(i < s["na"][:, None], s["acc"].long(), i)
    b = torch.arange(B, device="cuda")[:, None]
    src, dst = s["ctx"][:, None] + take, s["ctx"][:, None] + i
    ps, pd = (s["table"][b, (x // page).long()].long() for x in (src, dst))
    for pool in (s["kc"], s["vc"]):
        pool[pd, :, (dst % page).long()] = pool[ps, :, (src % page).long()]
    return zq, s["kc"], s["vc"], s["ctx"] + s["na"]


def _visible(s, slots):
    """[B, T, len(slots)]: what draft t of a sequence sees."""
    B, T = s["B"], s["T"]
    ctx = s["ctx"].long()[:, None, None]
    mask = s["mask"] if s["mask"] is not None else torch.ones((B, T), device="cuda", dtype=torch.int64)  # T = 1
    dl = (s["dl"].long() if s["dl"] is not None else torch.full((B,), T, device="cuda"))[:, None, None]
    u = slots[None, None] - ctx
    return (u < 0) | ((u < dl) & (((mask[:, :, None] >> u.clamp(0, 63)) & 1) == 1))


def _run_tree(s):
    B, T, Hq, Hkv, D, page = (s[x] for x in ("B", "T", "Hq", "Hkv", "D", "page"))
    if own:
        return _bsa().tree_attention(s["q"], s["kc"], s["vc"], s["table"], s["ctx"], draft_len=s["dl"],
                                     tree_mask=s["mask"], row_ptr=s["rp"], col_idx=s["ci"], out=s["o"], lse=s["lse"])
    G, P = Hq // Hkv, s["table"].shape[1]
    scale = 1.0 / math.sqrt(D)
    q = s["q"].float().reshape(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B * Hkv, T * G, D)
    # the listed (row, page) entries, every page of every row without a list
    if s["rp"] is None:
        row = torch.arange(B * Hkv, device="cuda").repeat_interleave(P)
        j = torch.arange(P, device="cuda").repeat(B * Hkv)
    else:
        row = torch.repeat_interleave(torch.arange(B * Hkv, device="cuda"), (s["rp"][1:] - s["rp"][:-1]).long(),
                                      output_size=s["ci"].numel())
        j = s["ci"].long()
    b, h = row // Hkv, row % Hkv
    end = s["ctx"].long() + (s["dl"].long() if s["dl"] is not None else T)
    slot = j[:, None] * page + torch.arange(page, device="cuda")
    held = slot < end[b][:, None]  # [E, page]
    pg = s["table"][b, j].long().clamp(min=0)
    K = s["kc"][pg, h].float()
    V = torch.where(held[..., None], s["vc"][pg, h].float(), 0.0)
    S = torch.bmm(q[row], K.transpose(1, 2)) * scale  # [E, T*G, page]
    allowed = torch.gather(_visible(s, torch.arange(P * page, device="cuda"))[b], 2,
                           slot[:, None].expand(-1, T, -1)) if s["rp"] is not None else \
        _visible(s, torch.arange(P * page, device="cuda")).reshape(B, T, P, page).permute(0, 2, 1, 3)[b, j]
    ok = (allowed & held[:, None]).repeat_interleave(G, dim=1)
    S = torch.where(ok, S, -math.inf)
    top = torch.full((B * Hkv, T * G), -math.inf, device="cuda")
    top.scatter_reduce_(0, row[:, None].expand(-1, T * G), S.amax(-1), "amax")
    base = torch.where(torch.isinf(top), 0.0, top)
    p = torch.exp(S - base[row][..., None])
    l = torch.zeros_like(top).index_add_(0, row, p.sum(-1))
    o = torch.zeros((B * Hkv, T * G, D), device="cuda").index_add_(0, row, torch.bmm(p, V))
    o = torch.where(l[..., None] > 0, o / l[..., None], 0.0)
    lse = torch.where(l > 0, base + torch.log(l), -math.inf)
    o = o.reshape(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    lse = lse.reshape(B, Hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, Hq)
    if s["dl"] is not None:
        on = torch.arange(T, device="cuda")[None] < s["dl"][:, None]
        o = torch.where(on[..., None, None], o, 0.0)
        lse = torch.where(on[..., None], lse, 0.0)
    return o.to(torch.bfloat16), lse


def _run_pages(s):
    page, kc, vc = s["page"], s["kc"], s["vc"]
    n_pages = s["ref"].shape[0]
    if own:
        bsa = _bsa()
        if s["call"] == "fork":
            bsa.cache_resize(s["table"], s["ref"], s["dst"], s["zero"], s["zero"], kc, vc)
            got = bsa.cache_fork(s["table"], s["ref"], s["src"], s["dst"], s["lens"], kc, vc)
            return s["table"], s["ref"], got, kc, vc
        # the fragmented state again (the pool's contents are not restored: the same pages move)
        s["table"].copy_(s["table0"])
        s["ref"].copy_(s["ref0"])
        new = bsa.cache_compact(s["table"], s["ref"], kc, vc)
        return s["table"], s["ref"], new, kc, vc
    if s["call"] == "fork":
        src, dst, lens = s["src"].long(), s["dst"].long(), s["lens"].long()
        P = s["table"].shape[1]
        j = torch.arange(P, device="cuda")[None]
        # the lost beams' pages go back; entry -1 counts in a place of its own
        lost = s["table"][dst].long()
        ref = torch.zeros(n_pages + 1, device="cuda", dtype=torch.int64)
        ref[:n_pages] = s["ref"]
        ref.index_add_(0, torch.where(lost < 0, n_pages, lost).reshape(-1), torch.full((lost.numel(),), -1, device="cuda"))
        free = torch.argsort((ref[:n_pages] != 0).to(torch.int8), stable=True)
        full, part = lens // page, lens % page
        # the pages to take in order, those of sequences that need none behind them
        spare = torch.argsort((part == 0).to(torch.int8), stable=True)
        fresh = torch.empty_like(dst).scatter_(0, spare, free[:dst.numel()])
        old = s["table"][src].long()
        row = torch.where(j < full[:, None], old, -1)
        row = torch.where((j == full[:, None]) & (part > 0)[:, None], fresh[:, None], row)
        ref.index_add_(0, torch.where(row < 0, n_pages, row).reshape(-1), torch.ones(row.numel(), device="cuda", dtype=torch.int64))
        s["table"][dst] = row.int()
        s["ref"].copy_(ref[:n_pages])
        # partial pages: their kept rows, or (no partial page) the new page onto itself
        a = torch.where(part > 0, old.gather(1, full[:, None].clamp(max=P - 1))[:, 0], fresh).clamp(min=0)
        keep = (torch.arange(page, device="cuda")[None] < part[:, None])[None, :, None, :, None]
        for pool in (kc, vc):
            pool[:, fresh] = torch.where(keep, pool[:, a], pool[:, fresh])
        return s["table"], s["ref"], torch.ones_like(s["dst"]), kc, vc
    s["table"].copy_(s["table0"])
    s["ref"].copy_(s["ref0"])
    live = s["ref"] > 0
    n_live = live.sum()
    i = torch.arange(n_pages, device="cuda")
    mover, hole = (live & (i >= n_live)).nonzero()[:, 0], (~live & (i < n_live)).nonzero()[:, 0]
    for pool in (kc, vc):
        pool[:, hole] = pool[:, mover]
    new = torch.where(live, i, -1)
    new[mover] = hole
    t = s["table"].long()
    s["table"].copy_(torch.where(t >= 0, new[t.clamp(min=0)], -1))
    s["ref"][hole] = s["ref"][mover]
    s["ref"][mover] = 0
    return s["table"], s["ref"], new.int(), kc, vc


# ------------------------------------------------------------------ work
def work(c):
    D = c.get("D")
    if c["op"] == "norm_rope":
        tok, Hq, Hkv, H2 = c["B"] * c["N"], c["Hq"], c["Hkv"], c["Hkv"] * c["rep"]
        if not c["grad"]:
            return {"bytes": tok * D * 2 * (2 * Hq + 2 * Hkv + 2 * H2), "flops": 10 * tok * D * (Hq + Hkv)}
        x = (Hq + Hkv) if c["norm"] else 0
        return {"bytes": tok * D * 2 * (Hq + 2 * H2 + x + Hq + 2 * Hkv), "flops": 20 * tok * D * (Hq + Hkv)}
    if c["op"] == "append":
        tok = c["B"] * c["T"]
        moved = 2 * c["Hkv"] * 2 * tok // 2 if c["T"] > 1 else 0
        return {"bytes": tok * D * 2 * 2 * (c["Hq"] + 2 * c["Hkv"]) + moved * D * 2,
                "flops": 10 * tok * D * (c["Hq"] + c["Hkv"])}
    if c["op"] == "tree":
        n = c["ctx"] * (0.5625 if c["ragged"] else 1.0) + c["T"]
        if c["listed_pages"]:
            n = min(n, (c["listed_pages"] - 0.5) * c["page"])
        rows = c["B"] * c["T"] * c["Hq"]
        return {"bytes": int(2 * c["B"] * c["Hkv"] * n * D * 2 + rows * D * 4 + rows * 4),
                "flops": int(4 * rows * n * D)}
    row = c["layers"] * 2 * c["Hkv"] * D * 2
    if c["call"] == "fork":
        half = max(1, c["n"] // 2)
        return {"bytes": int(2 * half * 0.5 * c["page"] * row) + 8 * half * c["ctx"] // c["page"] + 64, "flops": 0}
    return {"bytes": int(2 * 0.4 * 0.6 * c["pages"] * c["page"] * row) + 16 * c["pages"], "flops": 0}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "append": _exact_append, "tree": _exact_tree,
            "pages": _exact_pages}[case["op"]](s)


def _turn(x, w, pos, s, gain, eps=1e-6):
    """x [tokens, H, D], pos [tokens]: norm, then each pair times gain * e^(i angle), as complex numbers."""
    x = x.to(torch.float64)
    if w is not None:
        x = w.to(torch.float64) * x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + eps)
    rd = s["rd"]
    ang = torch.outer(pos.to(torch.float64), s["inv_freq"])
    e = torch.polar(torch.full_like(ang, gain), ang)[:, None]
    if s["interleaved"]:
        z = torch.view_as_complex(x[..., :rd].reshape(*x.shape[:-1], rd // 2, 2).contiguous()) * e
        z = torch.view_as_real(z).reshape(*x.shape[:-1], rd)
    else:
        z = torch.complex(x[..., :rd // 2].contiguous(), x[..., rd // 2:rd].contiguous()) * e
        z = torch.cat([z.real, z.imag], -1)
    return torch.cat([z, x[..., rd:]], -1)


def _exact_norm_rope(s):
    B, N, Hq, Hkv, rep, D = (s[x] for x in ("B", "N", "Hq", "Hkv", "rep", "D"))
    x = s["qkv"]
    pos = s["pos"] if s["pos"] is not None else torch.arange(N, device="cuda").repeat(B, 1)
    if not s["grad"]:
        outs = [torch.empty((B, H, N, D), device="cuda", dtype=torch.float64) for H in (Hq, Hkv * rep, Hkv * rep)]
        step = 16384
        for b in range(B):
            for n in range(0, N, step):
                m = min(N, n + step)
                part = x[b, n:m]
                outs[0][b, :, n:m] = _turn(part[:, :Hq], s["qw"], pos[b, n:m], s, s["gain"]).transpose(0, 1)
                zk = _turn(part[:, Hq:Hq + Hkv], s["kw"], pos[b, n:m], s, s["gain"])
                for h in range(Hkv * rep):
                    outs[1][b, h, n:m] = zk[:, h // rep]
                    outs[2][b, h, n:m] = part[:, Hq + Hkv + h // rep]
        return tuple(outs)
    # gradients by autograd through the definition
    gq, gk = (torch.empty((B, N, H, D), device="cuda", dtype=torch.float64) for H in (Hq, Hkv))
    gv = s["dz"][2].to(torch.float64).reshape(B, Hkv, rep, N, D).sum(2).transpose(1, 2)
    gw = [None if w is None else torch.zeros(D, device="cuda", dtype=torch.float64) for w in (s["qw"], s["kw"])]
    step = 4096
    with torch.enable_grad():
        for b in range(B):
            for n in range(0, N, step):
                m = min(N, n + step)
                for k, (lo, hi, w, g, r) in enumerate(((0, Hq, s["qw"], gq, 1), (Hq, Hq + Hkv, s["kw"], gk, rep))):
                    leaf = x[b, n:m, lo:hi].to(torch.float64).requires_grad_()
                    wl = None if w is None else w.to(torch.float64).requires_grad_()
                    z = _turn(leaf, wl, pos[b, n:m], s, s["gain"])
                    dz = s["dz"][k][b, :, n:m].to(torch.float64).reshape(hi - lo, r, m - n, D).sum(1).transpose(0, 1)
                    z.backward(dz)
                    g[b, n:m] = leaf.grad
                    if w is not None:
                        gw[k] += wl.grad
    return gq, gk, gv, gw[0], gw[1]


def _exact_append(s):
    Hq, Hkv, T, page = s["Hq"], s["Hkv"], s["T"], s["page"]
    x = s["qkv"]
    zq = _turn(x[:, :Hq], s["qw"], s["pos"], s, 1.0)
    zk = _turn(x[:, Hq:Hq + Hkv], s["kw"], s["pos"], s, 1.0)
    kc, vc = s["kc"].to(torch.float64), s["vc"].to(torch.float64)
    table, ctx = s["table"].cpu().tolist(), s["ctx"].cpu().tolist()
    acc, na = s["acc"].cpu().tolist(), s["na"].cpu().tolist()
    zv = x[:, Hq + Hkv:].to(torch.float64)
    for b, c in enumerate(ctx):
        # the rows of this sequence's drafts, in the order that the slots end up holding
        order = list(range(T))
        if T > 1:
            order[:na[b]] = acc[b][:na[b]]
        at = [(table[b][(c + i) // page], (c + i) % page) for i in range(T)]
        pg, sl = torch.tensor([p for p, _ in at]), torch.tensor([i for _, i in at])
        tok = torch.tensor([b * T + u for u in order]).to(zk.device)
        kc[pg, :, sl] = zk[tok]
        vc[pg, :, sl] = zv[tok]
    if T == 1:
        return zq, kc, vc
    return zq, kc, vc, s["ctx"] + s["na"]


def _exact_tree(s):
    B, T, Hq, Hkv, D, page = (s[x] for x in ("B", "T", "Hq", "Hkv", "D", "page"))
    G = Hq // Hkv
    O = torch.zeros((B, T, Hq, D), device="cuda", dtype=torch.float64)
    L = torch.zeros((B, T, Hq), device="cuda", dtype=torch.float64)
    ctx, table = s["ctx"].cpu().tolist(), s["table"].cpu().tolist()
    rp = s["rp"].cpu().tolist() if s["rp"] is not None else None
    ci = s["ci"].cpu().tolist() if s["ci"] is not None else None
    mask = s["mask"].cpu().tolist() if s["mask"] is not None else None
    for b in range(B):
        n = T if s["dl"] is None else int(s["dl"][b])
        end = ctx[b] + n
        tree = torch.tensor([[u <= t if mask is None else bool((mask[b][t] >> u) & 1) for u in range(n)]
                             for t in range(n)], device="cuda")
        see_all = torch.cat([torch.ones((n, ctx[b]), dtype=torch.bool, device="cuda"), tree], 1)
        for h in range(Hkv):
            js = range(-(-end // page)) if rp is None else ci[rp[b * Hkv + h]:rp[b * Hkv + h + 1]]
            js = [j for j in js if j * page < end]
            pg = torch.tensor([table[b][j] for j in js], device="cuda", dtype=torch.long)
            slots = (torch.tensor(js, device="cuda", dtype=torch.long)[:, None] * page
                     + torch.arange(page, device="cuda")).reshape(-1)
            inside = slots < end
            K = s["kc"][pg, h].reshape(-1, D)[inside].to(torch.float64)
            V = s["vc"][pg, h].reshape(-1, D)[inside].to(torch.float64)
            see = see_all[:, slots[inside]]
            q = s["q"][b, :n, h * G:(h + 1) * G].to(torch.float64)
            S = torch.einsum("tgd,sd->tgs", q, K) / math.sqrt(D)
            S = S.masked_fill(~see[:, None], -math.inf)
            lse = torch.logsumexp(S, -1)
            w = torch.exp(S - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
            O[b, :n, h * G:(h + 1) * G] = w @ V
            L[b, :n, h * G:(h + 1) * G] = lse
    return O, L


def _exact_pages(s):
    page, n_pages = s["page"], s["ref"].shape[0]
    table, ref = s["table"].cpu().tolist(), s["ref"].cpu().tolist()
    kc, vc = s["kc"].clone(), s["vc"].clone()
    if s["call"] == "fork":
        free = iter([p for p in range(n_pages) if ref[p] == 0])
        for a, b, n in zip(s["src"].tolist(), s["dst"].tolist(), s["lens"].tolist()):
            for j in range(n // page):
                table[b][j] = table[a][j]
                ref[table[a][j]] += 1
            if n % page:
                p, o = next(free), table[a][n // page]
                table[b][n // page], ref[p] = p, 1
                for pool in (kc, vc):
                    pool[:, p, :, :n % page] = pool[:, o, :, :n % page]
        third = torch.ones_like(s["dst"])
    else:
        live = [p for p in range(n_pages) if ref[p]]
        holes = [p for p in range(len(live)) if not ref[p]]
        move = dict(zip([p for p in live if p >= len(live)], holes))
        new = [move.get(p, p) if ref[p] else -1 for p in range(n_pages)]
        table = [[new[p] if p >= 0 else -1 for p in row] for row in table]
        a, b = torch.tensor(list(move), dtype=torch.long), torch.tensor(list(move.values()), dtype=torch.long)
        for pool in (kc, vc):
            pool[:, b] = pool[:, a]
        for p, to in move.items():
            ref[to], ref[p] = ref[p], 0
        third = torch.tensor(new, dtype=torch.int32)
    return (torch.tensor(table, dtype=torch.int32), torch.tensor(ref, dtype=torch.int32), third,
            kc, vc)
