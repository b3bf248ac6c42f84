"""The smallest calls of the serving entry points and the edges of their
contracts that a device decides, on one GPU."""

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


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("lists", [False, True])
def test_an_empty_batch_passes_through_a_serving_step(bsa, lists):
    """No sequences, no tokens: every call of a step returns empty results and
    leaves the pools as they were."""
    kc = torch.randn(4, 2, 64, 64, device="cuda").bfloat16()
    vc, k0 = kc + 1, kc.clone()
    none, table = i32(), torch.empty(0, 5, dtype=torch.int32, device="cuda")
    ref = torch.zeros(4, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    f, w = bsa.rope_inv_freq(64), torch.ones(64, device="cuda")
    for fn in (bsa.cache_resize, bsa.cache_fork):
        assert fn(table, ref, none, none, none, kc, vc).shape == (0,)
    q = bsa.cache_append(x, x[:, :2], x[:, :2], kc, vc, table, none, none, f, q_weight=w, k_weight=w)
    assert q.shape == (0, 4, 64)
    kw = dict(row_ptr=i32(0), col_idx=none) if lists else {}
    o, lse = bsa.tree_attention(q.view(0, 3, 4, 64), kc, vc, table, none, **kw)
    assert o.shape == (0, 3, 4, 64) and o.dtype == torch.bfloat16 and lse.shape == (0, 3, 4)
    n = bsa.cache_accept(kc, vc, table, none, torch.empty(0, 3, dtype=torch.int32, device="cuda"), none)
    assert n.shape == (0,) and n.dtype == torch.int32
    assert torch.equal(kc, k0) and bsa.device_error() == 0
    with pytest.raises(bsa.BsaError):  # a token of no sequence
        y = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
        bsa.cache_append(y, y, y, kc, vc, table, i32(0), i32(0), f)


@pytest.mark.parametrize("page,D", [(64, 128), (128, 64)])
def test_two_tokens_of_one_slot_leave_pieces_of_either(bsa, page, D):
    """No order among them, but nothing of a third row and no other slot touched."""
    n, H = 300, 3
    g = torch.Generator(device="cuda").manual_seed(page)
    x = torch.randn(n, 4 + 2 * H, D, generator=g, device="cuda").bfloat16()
    seq = torch.arange(n, device="cuda", dtype=torch.int32) % 3
    slot = torch.arange(n, device="cuda", dtype=torch.int32) // 3
    table = torch.arange(3 * 4, device="cuda", dtype=torch.int32).view(3, 4)
    f, w = bsa.rope_inv_freq(D), torch.rand(D, generator=g, device="cuda")

    def append(rows, seq, slot, pools):
        y = x[rows]
        bsa.cache_append(y[:, :4], y[:, 4:4 + H], y[:, 4 + H:], *pools, table, seq[rows], slot[rows], f,
                         positions=torch.arange(n, device="cuda", dtype=torch.int32)[rows], q_weight=w, k_weight=w)
        return pools

    pools = lambda: [torch.zeros(12, H, page, D, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    one, other = [r for r in range(n) if r != 250], [r for r in range(n) if r != 10]
    seq[250], slot[250] = seq[10], slot[10]
    both = append(list(range(n)), seq, slot, pools())
    for got, a, b in zip(both, append(one, seq, slot, pools()), append(other, seq, slot, pools())):
        pieces = [t.view(12, H, page, D // 8, 8) for t in (got, a, b)]
        from_a, from_b = (pieces[0] == pieces[1]).all(-1), (pieces[0] == pieces[2]).all(-1)
        assert (from_a | from_b).all()
        apart = ~(pieces[1] == pieces[2]).all(-1)
        assert int(apart.sum()) == H * D // 8  # the two tokens' slot, nothing else
    assert bsa.device_error() == 0


@pytest.mark.parametrize("page", [64, 128])
def test_listed_rows_hold_at_most_max_pages_entries(bsa, page):
    """Lists of a fixed width: up to max_pages entries those outside the table are
    skipped and reported; a longer row is malformed and counts as empty."""
    from test_gpu_tree import Case
    c = Case(2, 2, 4, 2, 64, page, [5 * page - 9, 3 * page], lists=lambda b, h, held, g: list(range(held)), seed=page)
    P = c.table.shape[1]
    held = [int((c.table[b] >= 0).sum()) for b in range(2)]
    rows = [list(range(held[r // 2])) for r in range(4)]

    def lists(rows):
        c.rp = torch.tensor([0] + [len(x) for x in rows]).cumsum(0).int()
        c.ci = torch.tensor([j for x in rows for j in x], dtype=torch.int32)

    pad = lambda x, n: x + [-1] * (n - len(x))
    lists([pad(x, P) for x in rows])
    c.check(*c.run(bsa))
    assert bsa.device_error() == 2
    lists([pad(rows[0], P), pad(rows[1], P + 1), rows[2], pad(rows[3], P + 5)])
    o, lse = c.run(bsa)
    assert bsa.device_error() == 2 | 4
    lists([pad(rows[0], P), [], rows[2], []])
    c.check(o, lse)
    assert (o[0, :, 2:] == 0).all() and torch.isneginf(lse[0, :, 2:]).all()
