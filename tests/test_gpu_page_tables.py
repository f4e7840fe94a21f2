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


@pytest.mark.parametrize("indptr,hkv", [
    ((0, 600, 300, 900), 2),                         # two kernels
    ((0, 5000, 2000, 2100, 7000), 1),
    ((0, 3000, 100) + (3100,) * 158, 1),             # one kernel, scores in the workspace
    ((0, 500, 100, 700) + (700,) * 157, 1),          # and in shared memory
], ids=["600", "5000", "160 of 3000", "160 of 600"])
def test_an_indptr_that_decreases(indptr, hkv):
    """Reported; the sequence that it ends before it begins selects nothing, and
    those that it makes overlap select their own pages or nothing."""
    ptr = torch.tensor(indptr, dtype=torch.int32)
    n = max(indptr)
    q, box, ids = _inputs(len(ptr) - 1, n, 2 * hkv, hkv, 128, n)
    sel, status = _select(q, box, ptr, ids, 33, 0)
    assert status == pkx.PKX_EDEVICE
    for b in range(len(ptr) - 1):
        if ptr[b + 1] < ptr[b]:
            assert (sel[b] == -1).all()
            continue
        want = R.select(q[b:b + 1], box, ptr[b:b + 2], ids, 33, 1, 1)[0]
        assert torch.equal(sel[b], want) or (sel[b] == -1).all()
