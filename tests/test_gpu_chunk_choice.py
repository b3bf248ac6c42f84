"""Which kernels a mixed batch is given follows the longest context the caller names,
not the width of a page table that is as wide as the longest context there may be."""

import pytest
import torch

from test_gpu_chunk import Case, both, bsa  # noqa: F401

pytestmark = pytest.mark.gpu

CTX = [900, 0, 333, 64, 1000, 512, 7, 640]
NEW = [1, 60, 1, 1, 2, 1, 1, 1]


def table_for(c, slots):
    """The case's sequences under a table for that many slots."""
    t = c.cache.table
    wide = torch.full((t.shape[0], slots // c.cache.page), -1, dtype=torch.int32)
    wide[:, :t.shape[1]] = t
    return wide.cuda()


@both
@pytest.mark.parametrize("D,page,window", [(128, 64, 0), (64, 128, 200)])
def test_a_wide_table_changes_nothing(bsa, D, page, window, q8):  # noqa: F811
    """The same bits as under a table as wide as the contexts, which is one kernel's work."""
    c = Case(CTX, NEW, 32, 8, D, page, q8, window, 3 if window else 0)
    assert not any(c.short)
    (q, k, v, table, ctx), more = c.args()
    o, lse = bsa.chunk_attention(q, k, v, table, ctx, **more)
    c.check(o, lse)
    wide = table_for(c, 131072)
    o2, lse2 = bsa.chunk_attention(q, k, v, wide, ctx, max_context=max(a + n for a, n in zip(CTX, NEW)), **more)
    assert bsa.device_error() == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@both
@pytest.mark.parametrize("max_context", [1, 100, 131072, 2 ** 31 - 1])
def test_a_wrong_bound_is_right_all_the_same(bsa, max_context, q8):  # noqa: F811
    c = Case(CTX, NEW, 32, 8, 128, 64, q8)
    (q, k, v, table, ctx), more = c.args()
    o, lse = bsa.chunk_attention(q, k, v, table_for(c, 131072), ctx, max_context=max_context, **more)
    assert bsa.device_error() == 0
    c.short = [max_context >= 131072 and n * 4 <= 16 for n in NEW]
    c.check(o, lse)


@both
def test_single_tokens_take_no_notice(bsa, q8):  # noqa: F811
    """One token a sequence is the short kernel's whatever the bound says."""
    c = Case([300, 5, 1000], [1, 1, 1], 8, 2, 128, 64, q8)
    (q, k, v, table, ctx), more = c.args(one=True)
    o, lse = bsa.chunk_attention(q, k, v, table, ctx, **more)
    c.check(o, lse)
    for m in (1, 10 ** 6):
        o2, lse2 = bsa.chunk_attention(q, k, v, table, ctx, max_context=m, **more)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    with pytest.raises((ValueError, RuntimeError)):
        bsa.chunk_attention(q, k, v, table, ctx, max_context=-1, **more)
    with pytest.raises((ValueError, RuntimeError, OverflowError)):
        bsa.chunk_attention(q, k, v, table, ctx, max_context=2 ** 31, **more)
    assert bsa.device_error() == 0


@both
@pytest.mark.parametrize("window,sinks", [(200, 4), (1000, 130)])
def test_a_window_bounds_the_work_too(bsa, window, sinks, q8):  # noqa: F811
    """However long the contexts may be, a few sequences under a window are one kernel's work."""
    c = Case(CTX, NEW, 32, 8, 128, 64, q8, window, sinks)
    (q, k, v, table, ctx), more = c.args()
    o, lse = bsa.chunk_attention(q, k, v, table, ctx, **more)
    c.check(o, lse)
    o2, lse2 = bsa.chunk_attention(q, k, v, table_for(c, 131072), ctx, **more)
    assert bsa.device_error() == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@both
def test_many_sequences_under_a_wide_window(bsa, q8):  # noqa: F811
    """Enough work for two kernels, by the window's width: single tokens to the short kernel's tolerance."""
    ctx, new = [(37 * b) % 300 for b in range(40)], [1, 1, 30, 1] * 10
    c = Case(ctx, new, 16, 16, 64, 64, q8, 4000, 4)
    (q, k, v, table, ctx), more = c.args()
    o, lse = bsa.chunk_attention(q, k, v, table_for(c, 131072), ctx, **more)
    assert bsa.device_error() == 0
    c.short = [n == 1 for n in new]
    c.check(o, lse)
