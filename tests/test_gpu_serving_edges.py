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
