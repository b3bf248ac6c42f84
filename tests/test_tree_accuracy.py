"""How exact the weights of tree_attention are: a bound close enough that the low
part of P shows, which is shown on the CPU to fail without it (planted in the
64-bit reference).

O = sum p v / sum p, A = sum p |v| / sum p.  The scores are exact here: q and k
hold integers of at most 3, a score is an integer below 2^24 times a scale of
2^-3, whatever the order of its sum.  What is left:
  exponent   x = s * scale * log2 e - reference: the factor is off by 2^-24 of
             itself, the sum by 2^-24 of x; the same reference stands in
             numerator and denominator.  2^x is off by 2^-22.  A weight's
             relative error: e = ln 2 * (2 |s| scale log2 e + |x|) 2^-24 + 2^-22
  P          a high and a low bf16 part: 2^-8 * 2^-8 = 2^-16 of a weight
  sums       n = 2 * slots / 16 products into an accumulator, in part through
             copies and parts of rows that are added once more (32 covers
             them), off by 2^-23 of at most A each; the sum of the weights by
             slots / 2 additions of 2^-24
  O: sum p |v| (2 e) / sum p + A (2^-16 + (slots / 8 + 32 + slots / 4) 2^-23) + |O| 2^-8
     (its own rounding)
"""

import numpy as np
import pytest
import torch

from test_gpu_tree import Case


@pytest.fixture(scope="module")
def bsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_flashattention_bsa_gb300 import build
    build.build()
    import block_sparse_flashattention_bsa_gb300 as m
    m.device_error()
    return m


SCALE = 0.125
SHAPES = [(1, 4, 1), (4, 16, 2), (8, 16, 2), (3, 43, 1), (16, 16, 2), (40, 4, 1)]  # T, Hq, Hkv: 4 to 160 rows a head
CTX = [0, 30, 64, 150, 127]


def integers(T, Hq, Hkv, D, page, ctx=CTX, lists=None):
    """A case of whole numbers in q and k."""
    c = Case(len(ctx), T, Hq, Hkv, D, page, ctx, seed=T + Hq + D + page, scale=SCALE, lists=lists)
    g = torch.Generator().manual_seed(D + T)
    draw = lambda shape: torch.randint(-3, 4, shape, generator=g).bfloat16()
    c.q = draw(c.q.shape)
    c.kc = torch.where(c.kc.isnan(), c.kc, draw(c.kc.shape))
    return c


def worst(c, o, p_parts=None):
    """Largest error of O in units of the bound; p_parts: P as that many bf16
    parts in place of the given O (rounded once to bf16)."""
    G, most = c.Hq // c.Hkv, 0.0
    for b in range(c.B):
        end = c.ctx[b] + c.T
        for h in range(c.Hkv):
            slots = torch.arange(end)
            if c.rp is not None:
                r = b * c.Hkv + h
                on = set(c.ci[c.rp[r]:c.rp[r + 1]].tolist())
                slots = torch.tensor([s for s in range(end) if s // c.page in on], dtype=torch.long)
            pg = c.table[b, slots // c.page].long()
            K, V = (x[pg, h, slots % c.page].double() for x in (c.kc, c.vc))
            bits = [int(x) & (2 ** 64 - 1) for x in c.mask[b]]
            see = torch.tensor([[s < c.ctx[b] or bits[t] >> (s - c.ctx[b]) & 1 for s in slots.tolist()]
                                for t in range(c.T)], dtype=torch.bool).view(c.T, 1, len(slots))
            S = torch.einsum("tgd,sd->tgs", c.q[b, :, h * G:(h + 1) * G].double(), K) * SCALE
            S = S.masked_fill(~see, -np.inf)
            top = S.amax(-1, keepdim=True) if len(slots) else torch.zeros(c.T, G, 1, dtype=torch.float64)
            top = top.masked_fill(top.isinf(), 0.0)  # rows that see nothing
            p = torch.exp(S - top)
            l = p.sum(-1, keepdim=True).clamp_min(1e-300)
            O, A = p @ V / l, p @ V.abs() / l
            if p_parts:
                q, rest = torch.zeros_like(p), p.float()
                for _ in range(p_parts):
                    q, rest = q + rest.bfloat16().double(), rest - rest.bfloat16().float()
                got = (q @ V / l).float().bfloat16().double()
            else:
                got = o[b, :, h * G:(h + 1) * G].detach().cpu().double()
            x = (S - top).abs().masked_fill(~see, 0.0) + 2 * S.abs().masked_fill(~see, 0.0)
            e = x * 2.0 ** -24 + 2.0 ** -22  # ln 2 * log2 e = 1
            n = len(slots) / 8 + 32 + len(slots) / 4
            tol = (p * 2 * e) @ V.abs() / l + A * (2.0 ** -16 + n * 2.0 ** -23) + O.abs() * 2.0 ** -8 + 1e-30
            assert torch.isfinite(got).all()
            most = max(most, ((got - O).abs() / tol).max().item())
    return most


@pytest.mark.parametrize("T,Hq,Hkv", SHAPES)
@pytest.mark.parametrize("D", [64, 128])
def test_the_bound_tells_one_part_from_two(D, T, Hq, Hkv):
    c = integers(T, Hq, Hkv, D, 64)
    assert worst(c, None, p_parts=2) <= 1
    assert worst(c, None, p_parts=1) > 1.5


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hkv", SHAPES)
@pytest.mark.parametrize("page", [64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_weights_are_exact(bsa, D, page, T, Hq, Hkv):
    """Every layout of rows (four splits, copies, neither, several tiles), items
    that are cut and that are not."""
    c = integers(T, Hq, Hkv, D, page)
    assert worst(c, c.run(bsa)[0]) <= 1
    c = integers(T, Hq, Hkv, D, page, CTX * 8,
                 lists=lambda b, h, held, g: torch.randperm(held, generator=g)[:max(1, held - h % 2)].tolist())
    assert worst(c, c.run(bsa)[0]) <= 1 and bsa.device_error() == 0
