"""GPU tests of select_pages over page tables that are slices of a larger one, or
broken: each sequence's selection is its own whatever stands before it."""
import pytest
import torch

import step_reference as R
from paged_kv_extend_gb300 import pkx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _inputs(batch, n, hq, hkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randperm(n + 3, generator=g)[:n].to(torch.int32)
    a, b = (torch.randn(n + 3, hkv, d, generator=g).bfloat16() for _ in range(2))
    box = torch.stack([torch.minimum(a, b), torch.maximum(a, b)], 2)
    return torch.randn(batch, hq, d, generator=g).bfloat16(), box, ids


def _select(q, box, indptr, ids, top, fill):
    """With every byte of the workspace set to ``fill`` before the call."""
    hkv = box.shape[1]
    ws = torch.full((pkx.select_pages_workspace_size(len(q), hkv, len(ids)),), fill, dtype=torch.uint8, device=DEV)
    sel, ws = pkx.select_pages(q.to(DEV), box.to(DEV), indptr.to(DEV), ids.to(DEV), top, 1, 1, workspace=ws)
    return sel.cpu(), pkx.workspace_status(ws)


@pytest.mark.parametrize("fill", [0, 255])
@pytest.mark.parametrize("indptr,n", [
    ((37, 637), 700),                      # inside a run of 32 entries
    ((64, 700), 700),                      # at the start of one
    ((5, 5, 5, 400, 401, 1300), 1400),     # empty sequences in front
    ((699, 1300, 1300), 1301),
    ((3, 3, 9, 12, 300), 300),             # one kernel
    ((31, 9000), 9031),
], ids=str)
def test_a_slice_of_a_page_table(indptr, n, fill):
    """The first sequence's pages begin past entry 0; entries before it, and
    behind the last sequence, are nobody's."""
    indptr = torch.tensor(indptr, dtype=torch.int32)
    q, box, ids = _inputs(len(indptr) - 1, n, 4, 2, 64, n)
    sel, status = _select(q, box, indptr, ids, 17, fill)
    assert torch.equal(sel, R.select(q, box, indptr, ids, 17, 1, 1))
    assert status == pkx.PKX_OK
