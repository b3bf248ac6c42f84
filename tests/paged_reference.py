"""Plain 64-bit counterparts of the paged-cache calls (torch, on the CPU), for the tests."""

import math

import torch

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def e4m3_values():
    """The 256 codes' values, from the format."""
    c = torch.arange(256)
    ex, mant = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(ex == 0, mant * 2.0 ** -9, (1 + mant / 8) * torch.pow(2.0, (ex - 7).double()))
    v = torch.where(c >= 128, -mag, mag)
    v[(c & 127) == 127] = math.nan
    return v


def quantise(y):
    """Codes and scale bytes (uint8) of rows y [..., D] (64 bits): nearest value, ties to the even code."""
    top = y.abs().amax(-1)
    e = torch.full(top.shape, -100, dtype=torch.long)
    for x in range(-100, 118):
        e = torch.where(top > 448 * 2.0 ** x, x + 1, e)
    z = (y / torch.pow(2.0, e.double())[..., None]).abs().clamp(max=448)
    v = e4m3_values()[:127]  # codes of values >= 0, ascending
    hi = torch.searchsorted(v, z).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = v[hi] - z, z - v[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code + torch.where(torch.signbit(y), 128, 0)).to(torch.uint8), (e + 127).to(torch.uint8)


def values(codes, scales):
    """64-bit values of rows of codes (uint8) with scale bytes (None: bf16 rows)."""
    if scales is None:
        return codes.double()
    return e4m3_values()[codes.long()] * torch.pow(2.0, scales.double() - 127)[..., None]


class Cache:
    """A cache of B sequences of lens[b] slots: random rows, everything else NaN; `layers` None: one layer."""

    def __init__(self, lens, Hkv, D, page, q8, seed=0, extra=2, spread=1.0, table_extra=1):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hkv, self.D, self.page, self.q8 = list(lens), Hkv, D, page, q8
        held = [-(-n // page) for n in lens]
        self.n_pages = sum(held) + extra
        order = torch.randperm(self.n_pages, generator=g).int()
        self.table = torch.full((len(lens), max([1, *held]) + table_extra), -1, dtype=torch.int32)
        shape = (self.n_pages, Hkv, page, D)
        self.k, self.v, self.ks, self.vs = None, None, None, None
        rows = [torch.full(shape, math.nan, dtype=torch.bfloat16) for _ in range(2)]
        at = 0
        for b, n in enumerate(lens):
            self.table[b, :held[b]] = order[at:at + held[b]]
            at += held[b]
            for j in range(held[b]):
                r = min(page, n - j * page)
                for x in rows:
                    size = torch.exp(spread * torch.randn(Hkv, r, 1, generator=g)) if spread != 1.0 else 1.0
                    x[int(self.table[b, j]), :, :r] = (torch.randn(Hkv, r, D, generator=g) * size).bfloat16()
        if not q8:
            self.k, self.v = rows
        else:
            for name, x in zip("kv", rows):
                bad = torch.isnan(x)
                codes, scales = quantise(torch.where(bad, 0, x).double())
                codes[bad] = 0x7F
                scales[bad[..., 0]] = 255
                setattr(self, name, codes)
                setattr(self, name + "s", scales)

    def device(self):
        """(k, v, table, keyword arguments of the scales) on the GPU."""
        if not self.q8:
            return self.k.cuda(), self.v.cuda(), self.table.cuda(), {}
        return (self.k.cuda().view(E4M3), self.v.cuda().view(E4M3), self.table.cuda(),
                dict(k_scale=self.ks.cuda().view(E8M0), v_scale=self.vs.cuda().view(E8M0)))

    def rows(self, b, h, slots):
        """64-bit K and V rows of slots (a tensor)."""
        pg, at = self.table[b, slots // self.page].long(), slots % self.page
        out = []
        for x, s in ((self.k, self.ks), (self.v, self.vs)):
            out.append(values(x[pg, h, at], None if s is None else s[pg, h, at]))
        return out


def attention(cache, q, q_ptr, ctx, window, sinks, scale):
    """64-bit O, LSE of every packed token, with A = sum p |v| and M = the largest scale * sum |q k|."""
    N, Hq, D = q.shape
    G = Hq // cache.Hkv
    O, A = (torch.zeros(N, Hq, D, dtype=torch.float64) for _ in range(2))
    L, M = (torch.zeros(N, Hq, dtype=torch.float64) for _ in range(2))
    for b in range(len(ctx)):
        r0, n = q_ptr[b], q_ptr[b + 1] - q_ptr[b]
        if n == 0:
            continue
        pos = torch.arange(ctx[b], ctx[b] + n)[:, None]
        slot = torch.arange(ctx[b] + n)[None]
        see = slot <= pos
        if window:
            see &= (slot > pos - window) | (slot < sinks)
        used = see.any(0).nonzero()[:, 0]
        see = see[:, used]
        for h in range(cache.Hkv):
            K, V = cache.rows(b, h, used)
            qh = q[r0:r0 + n, h * G:(h + 1) * G].double()
            S = torch.einsum("tgd,sd->tgs", qh, K) * scale
            big = torch.einsum("tgd,sd->tgs", qh.abs(), K.abs()) * scale
            S = S.masked_fill(~see[:, None], -math.inf)
            lse = torch.logsumexp(S, -1)
            p = torch.exp(S - lse[..., None])
            hs = slice(h * G, (h + 1) * G)
            O[r0:r0 + n, hs], A[r0:r0 + n, hs] = p @ V, p @ V.abs()
            L[r0:r0 + n, hs] = lse
            M[r0:r0 + n, hs] = big.masked_fill(~see[:, None], 0).amax(-1)
    return O, L, A, M


def check_attention(o, lse, ref, D, p_error):
    """Within the tolerances of test_gpu_chunk; returns the largest share of them that was used."""
    O, L, A, M = ref
    o, lse = o.cpu().double(), lse.cpu().double()
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    e = (D + 8) * M * 2.0 ** -24 + 2.0 ** -21
    tol = A * (p_error + 2 * e[..., None] + 2.0 ** -16) + O.abs() * 2.0 ** -8
    r = ((o - O).abs() / tol).amax().item()
    d = ((lse - L).abs() / (e + 2.0 ** -21 * (L.abs() + 1))).amax().item()
    assert r <= 1 and d <= 1, "O %.3g LSE %.3g of the tolerance" % (r, d)
    return max(r, d)
