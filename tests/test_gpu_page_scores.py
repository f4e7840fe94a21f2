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


def _reference(q, box, indptr, ids, top, first, last):
    """R.select with pages outside the bounds ranked behind all others."""
    hkv = box.shape[1]
    out = torch.full((len(q), hkv, top), -1, dtype=torch.int32)
    for b in range(len(q)):
        pages = ids[int(indptr[b]):int(indptr[b + 1])].long()
        n = len(pages)
        if n <= top:
            out[b, :, :n] = torch.arange(n, dtype=torch.int32)
            continue
        lost = (pages < 0) | (pages >= len(box))
        for h in range(hkv):
            s = R.scores(q[b].unflatten(0, (hkv, -1))[h], box[pages.masked_fill(lost, 0), h]).tolist()
            key = lambda p: (2, 0.0, p) if lost[p] else (0, 0.0, p) if s[p] != s[p] else (1, -s[p], p)
            rank = sorted(range(first, n - last), key=key)[:top - first - last]
            out[b, h] = torch.tensor(sorted([*range(first), *rank, *range(n - last, n)]))
    return out


SIZES = [  # pages of each sequence, selected pages
    ([50], (1, 20, 45)),
    ([300], (1, 100, 280)),              # two kernels, a warp selects
    ([900, 3], (7, 450, 850)),           # past the keys that its registers hold
    ([3000], (5, 1500, 2900)),           # 256 threads
    ([6000, 10], (33, 2500, 4096)),      # past theirs
    ([7000], (100, 4096)),               # 1024 threads
    ([20000], (100, 4096)),              # past theirs
    ([5000] + [20] * 159, (16, 4000)),   # one kernel, keys in the workspace
]


@pytest.mark.parametrize("pages,tops", SIZES, ids=lambda x: str(x[:2]))
def test_ties_zeros_nan_and_infinities(pages, tops):
    """Scores of a few values each: equal ones go to the lower page (-0 and +0 are
    equal), NaN ranks first, then +inf; -inf, the larger part, comes last."""
    indptr, ids, g = _table(pages)
    n, d, hkv = pages[0], 64, 1
    value = torch.randint(-1, 2, (sum(pages) + 3, hkv, 1, d), generator=g).bfloat16()
    value[..., 4:] = 0.0
    box = value.expand(-1, -1, 2, -1).contiguous()
    order = ids[torch.randperm(n, generator=g)].long()
    box[order[:3]] = -0.0
    box[order[3], 0, 1, 9] = float("nan")
    box[order[4], 0, 0, 2] = float("nan")
    box[order[5:8]] = 3.3e38
    few = order[8:8 + max(4, n * 2 // 5)]
    box[few] = -3.3e38  # finite; the sum is not
    q = torch.zeros(len(pages), 2, d, dtype=torch.bfloat16)
    q[:, 0, :8], q[:, 1, 2:6] = 1.0, 0.5
    s = R.scores(q[0], box[ids[:n].long(), 0])
    assert int((s == float("-inf")).sum()) == len(few) and int((s == float("inf")).sum()) == 3
    assert int(s.isnan().sum()) == 2 and len(s[s.isfinite()].unique()) < 40
    for top in tops:
        for first, last in ((0, 0), (1, 0)) if top > 1 else ((0, 0),):
            sel, status = _select(q, box, indptr, ids, top, first, last)
            assert status == pkx.PKX_OK
            assert torch.equal(sel, _reference(q, box, indptr, ids, top, first, last)), (top, first)


@pytest.mark.parametrize("pages,tops", SIZES, ids=lambda x: str(x[:2]))
def test_pages_outside_the_bounds_come_last(pages, tops):
    indptr, ids, g = _table(pages)
    n, top = pages[0], tops[-1]
    a, b = (torch.randn(sum(pages) + 3, 1, 64, generator=g).bfloat16() for _ in range(2))
    box = torch.stack([torch.minimum(a, b), torch.maximum(a, b)], 2)
    q = torch.randn(len(pages), 2, 64, generator=g).bfloat16()
    at = torch.randperm(n - 2, generator=g) + 1
    bad = ids.clone()
    lose = at[:n - top + 3]  # some of them have to be taken
    bad[lose[0::2]], bad[lose[1::2]] = -1, len(box)
    bad[lose[2]] = 2 ** 31 - 1
    sel, status = _select(q, box, indptr, bad, top, 1, 1)
    assert status == pkx.PKX_EDEVICE
    assert torch.equal(sel, _reference(q, box, indptr, bad, top, 1, 1))
    sel, status = _select(q, box, indptr, ids, top, 1, 1)
    assert status == pkx.PKX_OK and torch.equal(sel, R.select(q, box, indptr, ids, top, 1, 1))
    past = indptr.clone()
    past[-1] += 1
    sel, status = _select(q, box, past, ids, min(tops), 0, 0)
    assert status == pkx.PKX_EDEVICE and (sel[-1] == -1).all()
    want = _reference(q[:-1], box, indptr[:-1], ids, min(tops), 0, 0)
    assert torch.equal(sel[:-1], want)
