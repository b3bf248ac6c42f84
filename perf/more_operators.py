"""Cases, plain forms and 64-bit references of the operators of a quantised paged cache and of
the attention of new tokens over a paged cache.

Three families:

* ``append``: new tokens normed, rotated and written into a cache of 8-bit floating-point rows
  (e4m3), each row of a key head with a power of two of its own as its scale;
* ``read``: a range of slots of each sequence back as the contiguous head-major bf16 keys and
  values that the attention takes, key heads repeated, rows behind a sequence's end zero;
* ``attend``: attention of each sequence's new tokens (a chunk of a prompt, or one token) over
  its pages, causal, over all slots or over a sliding window and the first few tokens (sinks);
  bf16 pools or 8-bit ones.

``own`` False: elementary torch operations in 32 bits (64 for angles).  ``own`` True: the calls
of the package.
"""

from __future__ import annotations

import math
import random

import torch

own = False

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def _bsa():
    import block_sparse_flashattention_bsa_gb300 as bsa
    return bsa


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one stream: the launch counts
        dict(name="append_q8_one", op="append", B=1, T=1, ragged=False, Hq=32, Hkv=8, D=128, rd=128, page=128,
             ctx=2500, interleaved=False, norm=True),
        # the chunks of six prompts in one step
        dict(name="append_q8_prompts", op="append", B=6, T=4096, ragged=True, Hq=32, Hkv=8, D=128, rd=128, page=128,
             ctx=8192, interleaved=False, norm=True),
        # two long prefixes out of an 8-bit cache, for an attention with one key head per query head
        dict(name="read_q8_prefix", op="read", R=2, n=32768, q8=True, ragged=False, Hkv=8, rep=4, D=128, page=128),
        # a few short ragged prefixes out of a bf16 cache, padded to one length
        dict(name="read_ragged", op="read", R=5, n=1920, q8=False, ragged=True, Hkv=4, rep=1, D=64, page=64),
        # a chunk of a prompt behind a long cached prefix
        dict(name="chunk_2k", op="attend", mix="all", B=1, T=2048, ctx=32000, ragged=False, Hq=32, Hkv=8, D=128,
             page=128, q8=False, window=0, sinks=0),
        # the second half of a 16K prompt, 8-bit cache
        dict(name="chunk_8k_q8", op="attend", mix="all", B=1, T=8192, ctx=8192, ragged=False, Hq=32, Hkv=8, D=128,
             page=128, q8=True, window=0, sinks=0),
        # one step of a served batch: most sequences bring one token, some a piece of their prompt
        dict(name="chunk_mixed_q8", op="attend", mix="mixed", B=40, T=500, ctx=8192, ragged=True, Hq=40, Hkv=8, D=128,
             page=64, q8=True, window=0, sinks=0),
        # three short prompts of odd lengths, one key head per query head
        dict(name="chunk_odd", op="attend", mix="ragged", B=3, T=333, ctx=1000, ragged=True, Hq=16, Hkv=16, D=64,
             page=64, q8=False, window=0, sinks=0),
        # a chunk under a sliding window with four sinks
        dict(name="window_chunk", op="attend", mix="all", B=1, T=8192, ctx=16000, ragged=False, Hq=16, Hkv=2, D=64,
             page=64, q8=False, window=1024, sinks=4),
        # one token of each sequence under a window, long contexts
        dict(name="window_decode_q8", op="attend", mix="all", B=64, T=1, ctx=32768, ragged=True, Hq=32, Hkv=8, D=128,
             page=128, q8=True, window=4096, sinks=4),
        # one token of each sequence of a served batch, ragged contexts, 8-bit cache
        dict(name="decode_q8", op="attend", mix="all", B=96, T=1, ctx=8192, ragged=True, Hq=32, Hkv=8, D=128, page=128,
             q8=True, window=0, sinks=0),
        # one token of one stream, short context: latency
        dict(name="decode_q8_one", op="attend", mix="all", B=1, T=1, ctx=1500, ragged=False, Hq=16, Hkv=2, D=64,
             page=64, q8=True, window=0, sinks=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["append", "read", "attend", "attend", "attend", "attend"])
    D, page = rng.choice([64, 128]), rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 8, 16])
    if op == "append":
        B = _log(rng, 1, 200)
        T = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, 24576 // B))
        return dict(op=op, B=B, T=T, ragged=rng.random() < 0.5, Hq=Hkv * rng.choice([1, 2, 4, 5]), Hkv=Hkv, D=D,
                    rd=rng.choice([16, D // 2, D, D]), page=page, ctx=_log(rng, 1, 4000),
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.7)
    if op == "read":
        rep = rng.choice([1, 1, 2, 4, 5])
        R = _log(rng, 1, 16)
        most = 2 * 32768 * 32 * 128 // (R * Hkv * (rep + 1) * D)
        return dict(op=op, R=R, n=_log(rng, 1, min(65536, most)), q8=rng.random() < 0.6, ragged=rng.random() < 0.6,
                    Hkv=Hkv, rep=rep, D=D, page=page)
    G = rng.choice([1, 2, 4, 5, 8])
    Hq = Hkv * G
    q8, window, sinks = rng.random() < 0.5, 0, 0
    if rng.random() < 0.4:
        window, sinks = _log(rng, 1, 8192), rng.choice([0, 1, 4, 4, 130])
    mix = rng.choice(["all", "all", "ragged", "mixed", "one"])
    if mix == "one":  # decoding
        ctx = _log(rng, 1, 65536)
        B = _log(rng, 1, max(1, min(128, (54 if q8 else 27) * 8192 * 8 * 128 // (ctx * Hkv * D))))
        mix, T = "all", 1
    else:
        T, ctx = _log(rng, 1, 4096), _log(rng, 1, 32768)
        most = 8192 * 12288 * 32 * 128
        cost = lambda: T * (min(ctx + T, window + sinks + 64) if window else ctx + T) * Hq * D
        while cost() > most:
            T, ctx = T // 2, ctx // 2
        B = _log(rng, 1, max(1, min(48, most // cost(), 4 * 32768 * 8 * 128 // ((ctx + T) * Hkv * D),
                               8192 * 16 * 8 * 128 // (T * Hq * D))))
    return dict(op=op, mix=mix, B=B, T=T, ctx=ctx, ragged=rng.random() < 0.6, Hq=Hq, Hkv=Hkv, D=D, page=page, q8=q8,
                window=window, sinks=sinks)


def _lens(c):
    """(cached slots, new tokens) of each sequence: of the case, not of the seed."""
    r = random.Random("%d %d %d %d" % (c["B"], c["T"], c["ctx"], c["Hkv"]))
    B, T = c["B"], c["T"]
    ctx = [r.randint(c["ctx"] // 8, c["ctx"]) if c["ragged"] else c["ctx"] for _ in range(B)]
    mix = c.get("mix", "ragged" if c["ragged"] else "all")
    if mix == "all":
        new = [T] * B
    elif mix == "ragged":
        new = [r.randint(max(1, T // 4), T) for _ in range(B)]
    else:  # mixed: every tenth sequence brings a piece of its prompt, the others one token
        new = [r.randint(max(1, T // 4), T) if b % 10 == B % 10 or b == 0 else 1 for b in range(B)]
    return ctx, new


# ------------------------------------------------------------------ inputs
def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFF)
    return g


def _randn(shape, g, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32 if dtype == torch.float32 else dtype)
            * scale).to(dtype)


def _channels(D, g):
    """A few channels of keys and values are much larger than the others."""
    return torch.exp(0.5 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)


def _table(lens, page, extra, r):
    """A page table of sequences that hold `lens` slots, physical pages in random order."""
    held = [-(-n // page) for n in lens]
    order = list(range(sum(held) + extra))
    r.shuffle(order)
    t, at = torch.full((len(lens), max(1, max(held))), -1, dtype=torch.int32), 0
    for i, h in enumerate(held):
        t[i, :h] = torch.tensor(order[at:at + h], dtype=torch.int32)
        at += h
    return t, len(order)


def _pools(s, n_pages, Hkv, page, D, q8, g):
    for name in ("k", "v"):
        x = _randn((n_pages, Hkv, page, D), g) * _channels(D, g)
        if not q8:
            s[name + "c"], s[name + "s"] = x, None
            continue
        codes = torch.empty(x.shape, device="cuda", dtype=torch.uint8)
        scales = torch.empty(x.shape[:3], device="cuda", dtype=torch.uint8)
        for a in range(0, n_pages, 1024):
            codes[a:a + 1024], scales[a:a + 1024] = _quantised(x[a:a + 1024].float())
        s[name + "c"], s[name + "s"] = codes.view(E4M3), scales.view(E8M0)


def prepare(case, seed):
    return {"append": _prepare_append, "read": _prepare_read, "attend": _prepare_attend}[case["op"]](case, seed)


def _prepare_append(c, seed):
    g, r = _gen(seed), random.Random(seed)
    Hq, Hkv, D, page = (c[x] for x in ("Hq", "Hkv", "D", "page"))
    s = dict(c)
    ctx, new = _lens(c)
    t, n = _table([a + b for a, b in zip(ctx, new)], page, 3, r)
    s["table"] = t.cuda()
    _pools(s, n, Hkv, page, D, True, g)
    N = sum(new)
    s["qkv"] = _randn((N, Hq + 2 * Hkv, D), g) * _channels(D, g)
    i = torch.arange(c["rd"] // 2, dtype=torch.float64)
    s["inv_freq"] = (10000.0 ** (-2.0 * i / c["rd"])).cuda()
    s["qw"], s["kw"] = ((1 + 0.2 * _randn((D,), g, torch.float32)) if c["norm"] else None for _ in range(2))
    s["seq"] = torch.tensor([b for b, k in enumerate(new) for _ in range(k)], dtype=torch.int32).cuda()
    s["slot"] = torch.tensor([a + u for a, k in zip(ctx, new) for u in range(k)], dtype=torch.int32).cuda()
    return s


def _prepare_read(c, seed):
    g, r = _gen(seed), random.Random(seed)
    R, n, Hkv, D, page = (c[x] for x in ("R", "n", "Hkv", "D", "page"))
    s = dict(c)
    lr = random.Random("%d %d" % (R, n))
    lens = [lr.randint(max(1, n // 4), n) if c["ragged"] else n for _ in range(R)]
    t, n_pages = _table(lens, page, 2, r)
    s["table"] = t.cuda()
    _pools(s, n_pages, Hkv, page, D, c["q8"], g)
    order = list(range(R))
    r.shuffle(order)
    s["seq"] = torch.tensor(order, dtype=torch.int32).cuda()
    s["lens"] = torch.tensor([lens[i] for i in order], dtype=torch.int32).cuda()
    return s


def _prepare_attend(c, seed):
    g, r = _gen(seed), random.Random(seed)
    Hq, Hkv, D, page = (c[x] for x in ("Hq", "Hkv", "D", "page"))
    s = dict(c)
    ctx, new = _lens(c)
    t, n = _table([a + b for a, b in zip(ctx, new)], page, 2, r)
    s["table"] = t.cuda()
    _pools(s, n, Hkv, page, D, c["q8"], g)
    s["lens"] = (ctx, new)
    s["q"] = _randn((sum(new), Hq, D), g)
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32).cuda()
    at = [0]
    for k in new:
        at.append(at[-1] + k)
    s["q_ptr"] = None if max(new) == 1 else torch.tensor(at, dtype=torch.int32).cuda()
    return s


# ------------------------------------------------------------------ run
def run(state):
    return {"append": _run_append, "read": _run_read, "attend": _run_attend}[state["op"]](state)


def _quantised(y):
    """y [..., D] in 32 bits: e4m3 codes and the scales' biased exponents.  The scale is 2^e, e the
    smallest integer in [-100, 118] with max |y| <= 448 * 2^e."""
    m, k = torch.frexp(y.abs().amax(-1))
    e = (k - 9 + (m > 0.875)).clamp(-100, 118)
    codes = torch.ldexp(y, -e[..., None]).clamp(-448, 448).to(E4M3)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """fp32 values of rows of codes [..., D] with scales [...] (bf16 rows have none)."""
    x = codes.float()
    return x if scales is None else x * scales.float()[..., None]


def _normed(x, w, eps=1e-6):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w


def _rotated(y, ang, rd, interleaved):
    """y [N, H, D] in 32 bits, the pairs of its first rd values turned by ang [N, rd/2]."""
    c, sn = ang.cos().float()[:, None], ang.sin().float()[:, None]
    out = y.clone()
    if interleaved:
        a, b = y[..., 0:rd:2], y[..., 1:rd:2]
        out[..., 0:rd:2], out[..., 1:rd:2] = a * c - b * sn, b * c + a * sn
    else:
        a, b = y[..., :rd // 2], y[..., rd // 2:rd]
        out[..., :rd // 2], out[..., rd // 2:rd] = a * c - b * sn, b * c + a * sn
    return out


def _run_append(s):
    Hq, Hkv, rd, page = s["Hq"], s["Hkv"], s["rd"], s["page"]
    q, k, v = s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hkv], s["qkv"][:, Hq + Hkv:]
    if own:
        zq = _bsa().cache_append(q, k, v, s["kc"], s["vc"], s["table"], s["seq"], s["slot"], s["inv_freq"],
                                 q_weight=s["qw"], k_weight=s["kw"], interleaved=s["interleaved"], k_scale=s["ks"],
                                 v_scale=s["vs"])
        return zq, s["kc"], s["vc"], s["ks"], s["vs"]
    ang = s["slot"].double()[:, None] * s["inv_freq"]
    zq = _rotated(_normed(q, s["qw"]), ang, rd, s["interleaved"]).to(torch.bfloat16)
    zk = _rotated(_normed(k, s["kw"]), ang, rd, s["interleaved"])
    pg = s["table"][s["seq"].long(), (s["slot"] // page).long()].long()
    at = (s["slot"] % page).long()
    for pool, scales, y in ((s["kc"], s["ks"], zk), (s["vc"], s["vs"], v.float())):
        codes, e = _quantised(y)
        pool.view(torch.uint8)[pg, :, at] = codes
        scales.view(torch.uint8)[pg, :, at] = e
    return zq, s["kc"], s["vc"], s["ks"], s["vs"]


def _run_read(s):
    R, n, rep, page = s["R"], s["n"], s["rep"], s["page"]
    if own:
        return _bsa().cache_read(s["kc"], s["vc"], s["table"], s["seq"], s["lens"], n, kv_repeat=rep, k_scale=s["ks"],
                                 v_scale=s["vs"])
    slot = torch.arange(n, device="cuda")
    inside = slot[None] < s["lens"][:, None]  # [R, n]
    j = (slot // page).clamp(max=s["table"].shape[1] - 1)
    pg = s["table"][s["seq"].long()[:, None], j[None]].long().clamp(min=0)
    at = (slot % page)[None].expand(R, n)
    out = []
    for pool, scales in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
        if scales is None:
            x = pool[pg, :, at]  # [R, n, Hkv, D]
        else:
            x = _values(pool.view(torch.uint8)[pg, :, at].view(E4M3), scales.view(torch.uint8)[pg, :, at].view(E8M0))
        x = torch.where(inside[..., None, None], x, 0).to(torch.bfloat16)
        out.append(x.transpose(1, 2).repeat_interleave(rep, dim=1).contiguous())
    return tuple(out)


def _run_attend(s):
    Hq, Hkv, D, page, window, sinks = (s[x] for x in ("Hq", "Hkv", "D", "page", "window", "sinks"))
    if own:
        return _bsa().chunk_attention(s["q"], s["kc"], s["vc"], s["table"], s["ctx"], q_ptr=s["q_ptr"], window=window,
                                      sinks=sinks, k_scale=s["ks"], v_scale=s["vs"])
    G, scale = Hq // Hkv, 1.0 / math.sqrt(D)
    ctx, new = (torch.tensor(x) for x in s["lens"])
    # tiles of up to 64 tokens of one sequence: its number, its first token
    step = min(64, int(new.max()))
    n_tiles = (new + step - 1) // step
    b = torch.repeat_interleave(torch.arange(len(new)), n_tiles)
    first_tile = torch.cumsum(n_tiles, 0) - n_tiles
    t0 = (torch.arange(len(b)) - first_tile[b]) * step
    row0 = (torch.cumsum(new, 0) - new)[b] + t0
    most = int((ctx + new).max())
    b, t0, row0, ctx, new = (x.cuda() for x in (b, t0, row0, ctx, new))
    i = torch.arange(step, device="cuda")
    live = t0[:, None] + i < new[b][:, None]  # [X, step]
    row = torch.where(live, row0[:, None] + i, 0)
    pos = ctx[b][:, None] + t0[:, None] + i
    # the slots that a tile looks at: all, or the sinks and the union of its tokens' windows
    if window and sinks + window + step - 1 < most:
        j = torch.arange(sinks + window + step - 1, device="cuda")
        lo = (pos[:, 0] - window + 1).clamp(min=sinks)
        slot = torch.where(j < sinks, j, lo[:, None] + j - sinks)
    else:
        slot = torch.arange(most, device="cuda")[None].expand(len(b), most)
    end = (ctx + new)[b][:, None]
    inside = slot < end  # [X, W]
    see = inside[:, None] & (slot[:, None] <= pos[..., None])
    if window:
        see &= (slot[:, None] > pos[..., None] - window) | (slot[:, None] < sinks)
    pg = s["table"][b[:, None], torch.where(inside, slot // page, 0)].long().clamp(min=0)
    at = slot % page
    kv = []
    for pool, scales in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
        if scales is None:
            x = pool[pg, :, at].float()  # [X, W, Hkv, D]
        else:
            x = _values(pool.view(torch.uint8)[pg, :, at].view(E4M3), scales.view(torch.uint8)[pg, :, at].view(E8M0))
        kv.append(x.transpose(1, 2))
    X, W = slot.shape
    q = s["q"][row].float().reshape(X, step, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(X, Hkv, step * G, D)
    S = torch.matmul(q, kv[0].transpose(2, 3)).mul_(scale)
    S = S.reshape(X, Hkv, step, G, W).masked_fill_(~see[:, None, :, None], -math.inf)
    top = S.amax(-1, keepdim=True)
    base = torch.where(torch.isinf(top), 0.0, top)
    p = S.sub_(base).exp_()
    l = p.sum(-1, keepdim=True)
    v = torch.where(inside[:, None, :, None], kv[1], 0.0)
    o = torch.matmul(p.reshape(X, Hkv, step * G, W), v).reshape(X, Hkv, step, G, D)
    o = torch.where(l > 0, o / l, 0.0).permute(0, 2, 1, 3, 4).reshape(X, step, Hq, D)
    lse = (base + torch.log(l))[..., 0].permute(0, 2, 1, 3).reshape(X, step, Hq)
    return o[live].to(torch.bfloat16), lse[live]


# ------------------------------------------------------------------ work
def _seen(c):
    """Over all sequences: (slots that some new token sees, sum over the new tokens of what each sees)."""
    slots = pairs = 0
    w, k = c["window"], c["sinks"]
    for n, new in zip(*_lens(c)):
        end = n + new
        if not w:
            slots += end
            pairs += new * n + new * (new + 1) // 2
            continue
        slots += end - max(0, n - w + 1 - k)
        # a token at p sees min(p + 1, w) slots of its window and the sinks before it
        p = torch.arange(n, end, dtype=torch.int64)
        pairs += int((torch.clamp(p + 1, max=w) + torch.clamp(torch.clamp(p + 1 - w, min=0), max=k)).sum())
    return slots, pairs


def work(c):
    D, Hkv = c["D"], c["Hkv"]
    if c["op"] == "append":
        N = sum(_lens(c)[1])
        return {"bytes": N * (4 * D * c["Hq"] + 2 * Hkv * (2 * D + D + 1)), "flops": 10 * N * D * (c["Hq"] + 2 * Hkv)}
    row = D + 1 if c["q8"] else 2 * D
    if c["op"] == "read":
        lr = random.Random("%d %d" % (c["R"], c["n"]))
        n = sum(lr.randint(max(1, c["n"] // 4), c["n"]) if c["ragged"] else c["n"] for _ in range(c["R"]))
        return {"bytes": 2 * Hkv * (n * row + c["R"] * c["n"] * c["rep"] * 2 * D), "flops": 0}
    slots, pairs = _seen(c)
    N = sum(_lens(c)[1])
    return {"bytes": 2 * Hkv * slots * row + N * c["Hq"] * (4 * D + 4), "flops": 4 * c["Hq"] * D * pairs}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attend": _exact_attend}[case["op"]](s)


def _decoded(codes):
    """e4m3 codes (uint8) as 64-bit values, from the format: sign, four bits of exponent (bias 7), three of mantissa."""
    c = torch.arange(256)
    ex, mant = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(ex == 0, mant * 2.0 ** -9, (1 + mant / 8) * torch.pow(2.0, (ex - 7).double()))
    table = torch.where(c >= 128, -mag, mag)
    table[(c & 127) == 127] = math.nan
    return table.cuda()[codes.long()]


def _rounded(x):
    """64-bit x to the nearest e4m3 value (ties to the even mantissa)."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6)
    step = torch.pow(2.0, e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(s):
    Hq, Hkv, rd, page = s["Hq"], s["Hkv"], s["rd"], s["page"]
    x = s["qkv"].double()

    def turned(y, w):
        if w is not None:
            y = w.double() * y / torch.sqrt((y * y).sum(-1, keepdim=True) / y.shape[-1] + 1e-6)
        ang = torch.outer(s["slot"].double(), s["inv_freq"])[:, None]
        e = torch.polar(torch.ones_like(ang), ang)
        if s["interleaved"]:
            z = torch.view_as_complex(y[..., :rd].reshape(*y.shape[:-1], rd // 2, 2).contiguous()) * e
            z = torch.view_as_real(z).reshape(*y.shape[:-1], rd)
        else:
            z = torch.complex(y[..., :rd // 2].contiguous(), y[..., rd // 2:rd].contiguous()) * e
            z = torch.cat([z.real, z.imag], -1)
        return torch.cat([z, y[..., rd:]], -1)

    seq, slot = s["seq"].long(), s["slot"].long()
    pg = s["table"][seq, slot // page].long()
    out = [turned(x[:, :Hq], s["qw"])]
    scales = []
    for name, y in (("k", turned(x[:, Hq:Hq + Hkv], s["kw"])), ("v", x[:, Hq + Hkv:])):
        pool = _decoded(s[name + "c"].view(torch.uint8))
        sc = torch.pow(2.0, s[name + "s"].view(torch.uint8).double() - 127)
        top = y.abs().amax(-1)
        e = torch.ceil(torch.log2(top / 448))
        e = torch.where(top <= 448 * torch.pow(2.0, e - 1), e - 1, e)  # the logarithm of a power of two is rounded
        e = torch.where(top > 448 * torch.pow(2.0, e), e + 1, e).clamp(-100, 118)
        pool[pg, :, slot % page] = _rounded(y / torch.pow(2.0, e)[..., None])
        sc[pg, :, slot % page] = torch.pow(2.0, e)
        out.append(pool)
        scales.append(sc)
    return (*out, *scales)


def _exact_rows(s, b, slots):
    """64-bit key and value rows of `slots` (a tensor) of sequence b: [Hkv, n, D] each."""
    pg, at = s["table"][b, slots // s["page"]].long(), slots % s["page"]
    rows = []
    for name in ("k", "v"):
        if s[name + "s"] is None:
            x = s[name + "c"][pg, :, at].double()
        else:
            e = s[name + "s"].view(torch.uint8)[pg, :, at].double() - 127
            x = _decoded(s[name + "c"].view(torch.uint8)[pg, :, at]) * torch.pow(2.0, e)[..., None]
        rows.append(x.transpose(0, 1))
    return rows


def _exact_read(s):
    R, n, rep, Hkv, D = (s[x] for x in ("R", "n", "rep", "Hkv", "D"))
    out = [torch.zeros((R, Hkv * rep, n, D), device="cuda", dtype=torch.float64) for _ in range(2)]
    for i, (b, m) in enumerate(zip(s["seq"].tolist(), s["lens"].tolist())):
        for o, x in zip(out, _exact_rows(s, b, torch.arange(m, device="cuda"))):
            for h in range(Hkv * rep):
                o[i, h, :m] = x[h // rep]
    return tuple(out)


def _exact_attend(s):
    Hq, Hkv, D, window, sinks = (s[x] for x in ("Hq", "Hkv", "D", "window", "sinks"))
    G = Hq // Hkv
    O, L, at = [], [], 0
    for b, (n, new) in enumerate(zip(*s["lens"])):
        K, V = _exact_rows(s, b, torch.arange(n + new, device="cuda"))
        for t in range(0, new, 512):
            m = min(new, t + 512)
            pos = torch.arange(n + t, n + m, device="cuda")[:, None]
            # only the slots up to the last one seen, from the first one of a window without sinks
            lo = max(0, n + t - window + 1) if window and not sinks else 0
            slot = torch.arange(lo, n + m, device="cuda")[None]
            hide = slot > pos
            if window:
                hide |= (slot <= pos - window) & (slot >= sinks)
            q = s["q"][at + t:at + m].double().reshape(m - t, Hkv, G, D)
            o, l = [], []
            for h in range(Hkv):
                S = torch.einsum("tgd,sd->tgs", q[:, h], K[h, lo:n + m]) / math.sqrt(D)
                S = S.masked_fill(hide[:, None], -math.inf)
                lse = torch.logsumexp(S, -1)
                o.append(torch.exp(S - lse[..., None]) @ V[h, lo:n + m])
                l.append(lse)
            O.append(torch.stack(o, 1).reshape(m - t, Hq, D))
            L.append(torch.stack(l, 1).reshape(m - t, Hq))
        at += new
    return torch.cat(O), torch.cat(L)
