"""The weights' precision that the contract names for each row of a batch: by the rule
which kernel has the short sequences, restated here, at both of its thresholds (8-bit
pools 16 steps per SM, bf16 64) and on either side.

Tolerances are test_gpu_chunk's, with the weights' part by the rule: 2^-8, or 2^-16
(bf16 pools) and 2^-11 (8-bit).
"""

import pytest
import torch

from test_gpu_chunk import Case, both, bsa  # noqa: F401

pytestmark = pytest.mark.gpu


def tiles(slots):
    return -(-slots // 128)


def per_sm(q8):
    return (16 if q8 else 64) * torch.cuda.get_device_properties(0).multi_processor_count


def short_rows(c, Hkv, width, ptr=True, max_context=0):
    """Which sequences the kernel of the short ones works on (width: slots that the table is for)."""
    B, G = len(c.new), c.G
    if not ptr or sum(c.new) * G <= 16:
        return [n * G <= 16 for n in c.new]
    steps = min(tiles(width), tiles(max_context)) if max_context else tiles(width)
    if c.window:
        steps = min(steps, tiles(c.window) + 1 + tiles(c.sinks))
    return [n * G <= 16 and B > 1 and B * steps * Hkv > per_sm(c.cache.q8) for n in c.new]


def table_for(c, slots):
    t = c.cache.table
    wide = torch.full((t.shape[0], slots // c.cache.page), -1, dtype=torch.int32)
    wide[:, :t.shape[1]] = t
    return wide.cuda()


def run(bsa, c, Hkv, width=None, ptr=True, **kw):  # noqa: F811
    """The case's call, checked to what the contract says of each row."""
    (q, k, v, table, ctx), more = c.args(one=not ptr)
    if width:
        table = table_for(c, width)
    o, lse = bsa.chunk_attention(q, k, v, table, ctx, **more, **kw)
    assert bsa.device_error() == 0
    c.short = short_rows(c, Hkv, table.shape[1] * c.cache.page, ptr, kw.get("max_context", 0))
    c.check(o, lse)
    return o, lse


@both
@pytest.mark.parametrize("D", [64, 128])
def test_a_token_alone_and_beside_chunks(bsa, D, q8):  # noqa: F811
    """The same sequence alone, among single tokens, beside a chunk, and beside many: each to its own bound."""
    ctx = [700, 90, 1300, 255, 10, 64, 500, 2, 128, 400]
    new = [1, 200, 1, 1, 3, 1, 1, 130, 1, 1]
    mixed = Case(ctx, new, 16, 4, D, 64, q8)
    run(bsa, mixed, 4)
    assert not any(mixed.short)
    run(bsa, mixed, 4, width=1 << 20)
    assert [x for x, n in zip(mixed.short, new) if n * 4 <= 16] == [True] * 8
    alone = Case(ctx, new, 16, 4, D, 64, q8)
    (q, k, v, table, ctx_d), more = alone.args()
    sc = {x: more[x] for x in ("k_scale", "v_scale") if x in more}
    for b, n in enumerate(new):
        if n != 1:
            continue
        r = alone.q_ptr[b]
        o, lse = bsa.chunk_attention(q[r:r + 1].contiguous(), k, v, table[b:b + 1].contiguous(), ctx_d[b:b + 1], **sc)
        part = Case.__new__(Case)
        part.__dict__.update(alone.__dict__, q_ptr=[0, 1], new=[1], short=[True], ref=[x[r:r + 1] for x in alone.ref])
        part.check(o, lse)
    assert bsa.device_error() == 0


@both
@pytest.mark.parametrize("window", [0, 4000])
def test_both_sides_of_the_threshold(bsa, window, q8):  # noqa: F811
    """At the threshold one kernel (the bits of a bound of one slot), one step above it the finer weights."""
    ctx, new, Hkv = [300, 0, 64, 129, 1000, 17, 500, 31], [1, 40, 1, 2, 1, 1, 1, 4], 32
    c = Case(ctx, new, 2 * Hkv, Hkv, 64, 128, q8, window, 3 if window else 0)
    steps = per_sm(q8) // (len(ctx) * Hkv)
    one = run(bsa, c, Hkv, width=131072, max_context=1)
    assert not any(c.short)
    two = not window or tiles(window) + 1 + tiles(3) > steps  # else the window's own steps are too few
    for slots, short in ((128 * steps, False), (128 * steps + 1, two)):
        got = run(bsa, c, Hkv, width=131072, max_context=slots)
        assert any(c.short) == short
        if not short:
            assert torch.equal(got[0], one[0]) and torch.equal(got[1], one[1])


def test_8_bit_batches_between_the_thresholds(bsa):  # noqa: F811
    """More than 16 steps per SM, fewer than 64: 8-bit single tokens have the finer weights."""
    ctx, new = [(97 * b) % 1500 for b in range(24)], ([1, 1, 90, 1, 3, 1] * 4)
    c = Case(ctx, new, 16, 8, 128, 64, True)
    run(bsa, c, 8, width=4096)
    assert any(c.short) and not all(c.short)
    d = Case(ctx, new, 16, 8, 128, 64, False)
    run(bsa, d, 8, width=4096)
    assert not any(d.short)


@both
@pytest.mark.parametrize("D,page", [(64, 64), (128, 128)])
@pytest.mark.parametrize("G,count", [(1, 11), (1, 16), (1, 17), (4, 4), (5, 3), (8, 3), (16, 1)])
def test_few_rows_with_and_without_pointers(bsa, D, page, G, count, q8):  # noqa: F811
    """Up to 16 rows in all, q_ptr given: still the short form, as without it."""
    ctx = [0, 1, 62, 63, 64, 127, 128, 129, 300, 1000, 2049, 5, 640, 77, 256, 90, 31][:count]
    c = Case(ctx, [1] * count, 2 * G, 2, D, page, q8, seed=G)
    run(bsa, c, 2, ptr=False)
    assert all(c.short)
    run(bsa, c, 2)
    assert all(c.short) == (count * G <= 16)


@both
@pytest.mark.parametrize("count", [1024, 1025, 2100])
def test_more_sequences_than_a_launch_takes(bsa, count, q8):  # noqa: F811
    """Short sequences of several launches beside chunks, whose join is the last launch's."""
    ctx, new = [(53 * b) % 270 for b in range(count)], [0 if b % 11 == 3 else 40 if b % 97 == 5 else 1 for b in range(count)]
    c = Case(ctx, new, 8, 4, 64, 64, q8)
    run(bsa, c, 4, width=2048)
    assert any(c.short) and not all(c.short)
