"""GPU tests of decode attention over lists of more than 2^30 keys."""
import math

import pytest
import torch

from paged_kv_extend_gb300 import pkx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D = 64


def _pool(slots, needle):
    """Keys and values of zero but for one slot, whose logit with queries of one is
    64 (D ones, scale 1): exp(64) outweighs 2^31 other keys by 4e18."""
    k, v = (torch.zeros(slots, 1, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k[needle], v[needle] = 1.0, torch.arange(D, device=DEV).bfloat16()
    return k, v


def _check(o, lse, count, v):
    """`count` keys of logit 64 beside zeros.  The outputs are whole numbers that bf16
    holds: weights below 2e-9 for the rest, one rounding."""
    assert torch.equal(o, v.expand_as(o))
    want = 64 + math.log(count)
    assert ((lse.double() - want).abs() <= 1e-4).all()


@pytest.mark.parametrize("hq", [16, 17])
def test_an_own_list(hq):
    """16 query heads go to one kernel, 17 to another."""
    keys = (1 << 30) + 1000
    k, v = _pool(3, 2)
    idx = torch.zeros(keys, dtype=torch.int32, device=DEV)
    q = torch.ones(1, hq, D, dtype=torch.bfloat16, device=DEV)
    ptr = torch.tensor([0, keys], dtype=torch.int32, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    for at in (keys - 1, (1 << 30) + 2):
        idx[at] = 2
        o, lse = torch.zeros_like(q), torch.zeros(1, hq, device=DEV)
        ws = pkx.decode_attention_fwd_shared(q, o, k, v, ptr, idx, torch.zeros(1, dtype=torch.int32, device=DEV), none,
                                             sm_scale=1.0, lse=lse)
        assert pkx.workspace_status(ws) == pkx.PKX_OK
        _check(o, lse, 1, v[2])
        idx[at] = 0


@pytest.mark.parametrize("hq", [16, 17])
def test_selected_pages(hq):
    """4096 entries of 2^18 + 64 places; only the last one is of the page that holds
    the needle, in its last place."""
    page, top = (1 << 18) + 64, 4096
    k, v = _pool(2 * page, 2 * page - 1)
    ids = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    ptr, last = ids * 2, torch.full((1,), page, dtype=torch.int32, device=DEV)
    sel = torch.zeros(1, 1, top, dtype=torch.int32, device=DEV)
    sel[0, 0, -1] = 1
    q = torch.ones(1, hq, D, dtype=torch.bfloat16, device=DEV)
    o, lse = torch.zeros_like(q), torch.zeros(1, hq, device=DEV)
    ws = pkx.decode_attention_fwd_pages(q, o, k, v, ptr, ids, last, page, sel, sm_scale=1.0, lse=lse)
    assert pkx.workspace_status(ws) == pkx.PKX_OK
    _check(o, lse, 1, v[-1])


@pytest.mark.parametrize("hq", [16, 17])
def test_the_largest_page(hq):
    """One page of 2^31 - 4097 places, of which five are in use, outside the pool: its
    keys read as zero rows, and it is reported."""
    page = 2 ** 31 - 4097
    k, v = _pool(64, 0)
    one = torch.zeros(1, dtype=torch.int32, device=DEV)
    ptr = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    q = torch.ones(1, hq, D, dtype=torch.bfloat16, device=DEV)
    o, lse = torch.ones_like(q), torch.zeros(1, hq, device=DEV)
    ws = pkx.decode_attention_fwd_pages(q, o, k, v, ptr, one, one + 5, page, one.view(1, 1, 1), sm_scale=1.0, lse=lse)
    assert pkx.workspace_status(ws) == pkx.PKX_EDEVICE
    assert not o.any() and ((lse.double() - math.log(5)).abs() <= 1e-5).all()
