"""GPU tests of select_pages' scores: ties, zeros, NaN, -inf and pages outside the
bounds at every size of the selection kernels, and queries that hold NaN."""
import pytest
import torch

import step_reference as R
from paged_kv_extend_gb300 import pkx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _select(q, box, indptr, ids, top, first=0, last=0):
    on = [x.to(DEV) for x in (q, box, indptr, ids)]
    sel, ws = pkx.select_pages(*on, top, first, last)
    return sel.cpu(), pkx.workspace_status(ws)


def _table(pages, spare=3):
    g = torch.Generator().manual_seed(sum(pages))
    indptr = torch.tensor([0] + torch.tensor(pages).cumsum(0).tolist(), dtype=torch.int32)
    return indptr, torch.randperm(sum(pages) + spare, generator=g)[:sum(pages)].to(torch.int32), g


@pytest.mark.parametrize("pages", [[50], [600], [5000], [40] * 3])
@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_query_takes_its_own_kv_head(pages, d):
    """A NaN in any query head of a KV head makes all of its scores NaN, so that the
    lowest pages are selected; other KV heads and sequences select their own."""
    indptr, ids, g = _table(pages)
    top, hq, hkv = 12, 6, 2
    a, b = (torch.randn(sum(pages) + 3, hkv, d, generator=g).bfloat16() for _ in range(2))
    box = torch.stack([torch.minimum(a, b), torch.maximum(a, b)], 2)
    q = torch.randn(len(pages), hq, d, generator=g).bfloat16()
    want = R.select(q, box, indptr, ids, top, 1, 1)
    q[0, 4, d - 3] = float("nan")  # the second KV head's
    want[0, 1] = torch.tensor([*range(top - 1), pages[0] - 1])
    sel, status = _select(q, box, indptr, ids, top, 1, 1)
    assert status == pkx.PKX_OK and torch.equal(sel, want)
