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


@pytest.mark.parametrize("hq", [8, 34])
def test_decode_over_slices_of_larger_lists(hq):
    """Decode over selected pages and with a shared prefix, whose first sequence's entries
    begin past entry 0: the same bits as with the lists cut to size."""
    g = torch.Generator().manual_seed(hq)
    hkv, d, page = 2, 64, 16
    k, v = (torch.randn(60 * page, hkv, d, generator=g).bfloat16().to(DEV) for _ in range(2))
    q = torch.randn(3, hq, d, generator=g).bfloat16().to(DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    ids = torch.randperm(60, generator=g)[:57].to(torch.int32).to(DEV)
    slots = torch.randperm(60 * page, generator=g)[:900].to(torch.int32).to(DEV)

    def run(cut):
        at = 7 * (not cut)
        o, o2 = torch.empty_like(q), torch.empty_like(q)
        lse, lse2 = torch.empty(3, hq, device=DEV), torch.empty(3, hq, device=DEV)
        sel, ws = pkx.select_pages(q, box, i32(at, at + 20, at + 20, at + 45), ids[7:].contiguous() if cut else ids, 9)
        ws2 = pkx.decode_attention_fwd_pages(q, o, k, v, i32(at, at + 20, at + 20, at + 45),
                                             ids[7:].contiguous() if cut else ids, i32(5, 0, 16), page, sel, lse=lse)
        ws3 = pkx.decode_attention_fwd_shared(q, o2, k, v, i32(at, at + 300, at + 610, at + 880),
                                              slots[7:].contiguous() if cut else slots, i32(0, 2), i32(290), lse=lse2)
        assert all(pkx.workspace_status(w) == pkx.PKX_OK for w in (ws, ws2, ws3))
        return sel, o, lse, o2, lse2

    box = torch.zeros(60, hkv, 2, d, dtype=torch.bfloat16, device=DEV)
    pkx.update_page_bounds(k, box, torch.arange(60, dtype=torch.int32, device=DEV), page)
    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)
