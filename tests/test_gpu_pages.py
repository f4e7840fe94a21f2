"""GPU tests of page bounds, page selection and decode over selected pages."""
import random

import pytest
import torch

import step_reference as R
from paged_kv_extend_gb300 import pkx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _pool(g, slots, hkv, d, kv):
    return torch.randn(slots, hkv, d, generator=g).to(kv)


@pytest.mark.parametrize("kv", [torch.bfloat16, torch.float8_e4m3fn, torch.float8_e5m2], ids=str)
@pytest.mark.parametrize("hkv,d,page,n", [(1, 64, 1, 5), (3, 64, 16, 9), (8, 128, 64, 7), (2, 72, 130, 3)])
def test_bounds(hkv, d, page, n, kv):
    g = torch.Generator().manual_seed(page + d)
    total = n + 3
    k = _pool(g, total * page + 2, hkv, d, kv)
    ids = torch.randperm(total, generator=g)[:n].to(torch.int32)
    lens = torch.randint(1, page + 1, (n,), generator=g).to(torch.int32)
    lens[0] = page + 5  # held at the page size
    old = torch.full((total, hkv, 2, d), 7.0, dtype=torch.bfloat16)
    bad = torch.tensor([-1, total, int(ids[1]), 2 ** 31 - 1], dtype=torch.int32)
    bad_lens = torch.tensor([3, 3, 0, 1], dtype=torch.int32)
    out = pkx.update_page_bounds(k.to(DEV), old.to(DEV), torch.cat([ids, bad]).to(DEV), page,
                                 page_lens=torch.cat([lens, bad_lens]).to(DEV))
    assert torch.equal(out.cpu(), R.bounds(k, ids, lens, page, old))
    out = pkx.update_page_bounds(k.to(DEV), old.to(DEV), ids.to(DEV), page)
    assert torch.equal(out.cpu(), R.bounds(k, ids, torch.full_like(lens, page), page, old))


def test_bounds_of_strided_pools_nan_and_infinity():
    g = torch.Generator().manual_seed(5)
    both = torch.randn(64, 2, 4, 64, generator=g).bfloat16()
    both[3, 0, 1, 2], both[17, 0, 0, 0], both[40, 0, 3, 9] = float("nan"), float("inf"), float("-inf")
    ids = torch.arange(4, dtype=torch.int32)
    old = torch.zeros(4, 4, 2, 64, dtype=torch.bfloat16)
    out = pkx.update_page_bounds(both.to(DEV)[:, 0], old.to(DEV), ids.to(DEV), 16).cpu()
    want = R.bounds(both[:, 0], ids, torch.full((4,), 16), 16, old)
    assert torch.equal(out.isnan(), want.isnan()) and out[0, 1, :, 2].isnan().all()
    assert torch.equal(out.nan_to_num(9.0), want.nan_to_num(9.0))
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    assert torch.equal(pkx.update_page_bounds(both.to(DEV)[:, 0], old.to(DEV), none, 16).cpu(), old)


def _batch(g, pages, total=None):
    """Page table of sequences with these many pages each."""
    indptr = torch.tensor([0] + torch.tensor(pages).cumsum(0).tolist(), dtype=torch.int32)
    ids = torch.randperm(total or sum(pages) + 3, generator=g)[:sum(pages)].to(torch.int32)
    return indptr, ids


SELECT = [  # pages of each sequence, hq, hkv, d, top, first, last
    ([1], 1, 1, 64, 1, 0, 0),
    ([40, 0, 1, 17, 8], 12, 3, 64, 8, 1, 2),
    ([5, 300, 33], 32, 8, 128, 32, 1, 1),
    ([700, 3], 14, 2, 128, 129, 0, 3),
    ([9, 9], 4, 4, 128, 3, 2, 1),  # no room for others
    ([6000], 4, 1, 64, 500, 1, 1),  # past the keys held in registers (256 threads)
    ([20000], 2, 1, 64, 4000, 5, 6),  # and with 1024
    ([33] * 70, 128, 1, 64, 4, 0, 1),
    ([900, 3], 8, 2, 64, 40, 1, 1),  # a warp each, past the keys that it holds
    ([3000, 100], 8, 2, 128, 200, 2, 0),
    ([7000, 10, 10], 4, 1, 64, 300, 0, 1),
    ([5000] + [20] * 79, 2, 2, 128, 16, 1, 1),  # one kernel, keys in the workspace
    ([600, 31, 0, 64] * 20, 6, 2, 64, 33, 1, 2),
]


@pytest.mark.parametrize("case", SELECT, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[1:]}")
def test_selection_is_exact(case):
    pages, hq, hkv, d, top, first, last = case
    g = torch.Generator().manual_seed(sum(pages))
    indptr, ids = _batch(g, pages)
    a, b = (torch.randn(sum(pages) + 3, hkv, d, generator=g).bfloat16() for _ in range(2))
    box = torch.stack([torch.minimum(a, b), torch.maximum(a, b)], 2)
    q = torch.randn(len(pages), hq, d, generator=g).bfloat16()
    sel, ws = pkx.select_pages(q.to(DEV), box.to(DEV), indptr.to(DEV), ids.to(DEV), top, first, last)
    assert torch.equal(sel.cpu(), R.select(q, box, indptr, ids, top, first, last))
    assert pkx.workspace_status(ws) == pkx.PKX_OK


def test_ties_zeros_and_nan():
    """Equal scores go to the lower page (-0 and +0 are equal), NaN ranks first,
    -inf last; indices past kv_indptr's end are no candidates."""
    n, d = 50, 64
    box = torch.zeros(n + 2, 1, 2, d, dtype=torch.bfloat16)
    box[10:20] = 1.0
    box[3, 0, :, 0] = -0.0
    box[30, 0, 1, 4] = float("nan")
    box[31, 0, 0, :] = float("-inf")
    box[31, 0, 1, :] = float("-inf")
    q = torch.zeros(1, 2, d, dtype=torch.bfloat16)
    q[0, 0, :8] = 1.0
    indptr, ids = torch.tensor([0, n], dtype=torch.int32), torch.arange(n + 2, dtype=torch.int32)
    for top in (1, 5, 11, 12, 14, 45, 48, 49):
        sel, _ = pkx.select_pages(q.to(DEV), box.to(DEV), indptr.to(DEV), ids.to(DEV), top, 0, 0)
        assert torch.equal(sel.cpu(), R.select(q, box, indptr, ids, top, 0, 0)), top


def test_selection_reports_bad_pages_and_indptrs():
    d = 64
    box = torch.randn(8, 1, 2, d, device=DEV).bfloat16()
    q = torch.randn(2, 1, d, device=DEV).bfloat16()
    ids = torch.tensor([0, 1, -5, 3, 99, 2, 4, 5], dtype=torch.int32, device=DEV)
    ptr = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    sel, ws = pkx.select_pages(q, box, ptr(0, 5, 8), ids, 3, 0, 0)
    assert pkx.workspace_status(ws) == pkx.PKX_EDEVICE
    assert sel[0, 0].tolist() == [0, 1, 3] and sel[1, 0].tolist() == [0, 1, 2]
    for p in (ptr(0, 5, 4), ptr(0, 5, 9), ptr(-1, 2, 4)):
        sel, ws = pkx.select_pages(q, box, p, ids, 4, 0, 0, workspace=ws)
        assert pkx.workspace_status(ws) == pkx.PKX_EDEVICE
        assert (sel[0] == -1).all() or (sel[1] == -1).all()
    sel, ws = pkx.select_pages(q, box, ptr(0, 2, 4), ids[[0, 1, 5, 6]].contiguous(), 1, 0, 0, workspace=ws)
    assert pkx.workspace_status(ws) == pkx.PKX_OK
    sel, ws = pkx.select_pages(q, box, ptr(0, 0, 0), ids[:0], 2)
    assert (sel == -1).all() and pkx.workspace_status(ws) == pkx.PKX_OK


def _reference(case, q, k, v, indptr, ids, last, sel, scale, cap, ks, vs):
    hkv, page = k.shape[1], case["page"]
    o, size = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64)
    g = q.shape[1] // hkv
    for b in range(q.shape[0]):
        n = int(indptr[b + 1] - indptr[b])
        for h in range(hkv):
            slots = []
            for s in sel[b, h].tolist():
                if 0 <= s < n:
                    start = int(ids[int(indptr[b]) + s]) * page
                    slots += range(start, start + (int(last[b]) if s == n - 1 else page))
            rows = slice(h * g, (h + 1) * g)
            at = torch.tensor(slots, dtype=torch.int64)
            o[b, rows], lse[b, rows], size[b, rows] = R.attend(
                q[b, rows].double(), k.double()[at, h] * ks, v.double()[at, h] * vs, scale, cap)
    return o, lse, size


ATTEND = [  # keys of each sequence, page, hq, hkv, d, top, kv, cap
    dict(keys=[1], page=1, hq=1, hkv=1, d=64, top=1, kv=torch.bfloat16, cap=0.0),
    dict(keys=[700, 0, 1, 129, 40], page=16, hq=12, hkv=3, d=64, top=9, kv=torch.bfloat16, cap=0.0),
    dict(keys=[2000, 333], page=64, hq=32, hkv=8, d=128, top=20, kv=torch.bfloat16, cap=0.0),
    dict(keys=[500, 77], page=33, hq=14, hkv=2, d=128, top=7, kv=torch.bfloat16, cap=4.0),
    dict(keys=[900, 5, 64], page=32, hq=28, hkv=4, d=128, top=11, kv=torch.float8_e4m3fn, cap=0.0),
    dict(keys=[900, 5, 64], page=32, hq=8, hkv=1, d=64, top=11, kv=torch.float8_e5m2, cap=0.0),
    dict(keys=[5000], page=200, hq=128, hkv=1, d=64, top=25, kv=torch.bfloat16, cap=0.0),
    dict(keys=[4000, 0, 90], page=64, hq=34, hkv=2, d=128, top=60, kv=torch.float8_e4m3fn, cap=0.0),
    dict(keys=[4000, 31], page=16, hq=16, hkv=1, d=128, top=240, kv=torch.bfloat16, cap=2.0),
    dict(keys=[90, 3, 0, 41], page=16, hq=12, hkv=2, d=128, top=6, kv=torch.float8_e4m3fn, cap=0.0),  # one unit a head
    dict(keys=[90, 3, 0, 41], page=16, hq=26, hkv=2, d=64, top=5, kv=torch.float8_e5m2, cap=2.0),
    dict(keys=[3000, 9], page=24, hq=9, hkv=1, d=64, top=100, kv=torch.float8_e4m3fn, cap=0.0),
    dict(keys=[40] * 150, page=8, hq=4, hkv=2, d=128, top=3, kv=torch.bfloat16, cap=0.0),
]


def _attend_case(case, seed):
    r, g = random.Random(seed), torch.Generator().manual_seed(seed)
    pages = [-(-t // case["page"]) for t in case["keys"]]
    indptr, ids = _batch(g, pages)
    last = torch.tensor([t - (p - 1) * case["page"] if p else 0 for t, p in zip(case["keys"], pages)],
                        dtype=torch.int32)
    slots = (sum(pages) + 3) * case["page"]
    k, v = (_pool(g, slots, case["hkv"], case["d"], case["kv"]) for _ in range(2))
    q = torch.randn(len(pages), case["hq"], case["d"], generator=g).bfloat16()
    sel = torch.full((len(pages), case["hkv"], case["top"]), -1, dtype=torch.int32)
    for b, n in enumerate(pages):
        for h in range(case["hkv"]):
            pick = sorted(r.sample(range(n), min(n, case["top"])))
            sel[b, h, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
    return q, k, v, indptr, ids, last, sel


def _attend(case, q, k, v, indptr, ids, last, sel, ws=None):
    on = [x.to(DEV) for x in (q, k, v, indptr, ids, last, sel)]
    o = torch.full_like(on[0], float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device=DEV)
    ks, vs = (1.0, 1.0) if case["kv"] == torch.bfloat16 else (0.37, 1.9)
    ws = pkx.decode_attention_fwd_pages(on[0], o, on[1], on[2], on[3], on[4], on[5], case["page"], on[6], 0.11,
                                        case["cap"], lse=lse, k_scale=ks, v_scale=vs, workspace=ws)
    return o, lse, ws, (0.11, case["cap"], ks, vs)


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"{c['keys'][:3]}-{c['page']}-{c['hq']}/{c['hkv']}x{c['d']}")
def test_attention_over_selected_pages(case):
    args = _attend_case(case, 3)
    o, lse, ws, s = _attend(case, *args)
    assert pkx.workspace_status(ws) == pkx.PKX_OK
    R.check_attention(o, lse, _reference(case, *args, *s), case["cap"])


def test_attention_takes_any_selection():
    """Unordered entries, gaps and a page listed twice; numbers past the
    sequence's pages are left out and reported, a page outside the pool reads as
    zero rows."""
    case = dict(keys=[300, 100], page=16, hq=8, hkv=2, d=128, top=6, kv=torch.bfloat16, cap=0.0)
    q, k, v, indptr, ids, last, sel = _attend_case(case, 8)
    sel[0, 0] = torch.tensor([18, -1, 3, 3, -7, 0])
    sel[0, 1] = -1
    args = (q, k, v, indptr, ids, last, sel)
    o, lse, ws, s = _attend(case, *args)
    assert pkx.workspace_status(ws) == pkx.PKX_OK
    R.check_attention(o, lse, _reference(case, *args, *s))
    assert not o[0, 4:].any()
    sel[1, 1, 0] = 7  # has 7 pages
    o, lse, ws, s = _attend(case, *args, ws=ws)
    assert pkx.workspace_status(ws) == pkx.PKX_EDEVICE
    R.check_attention(o, lse, _reference(case, *args, *s))
    sel[1, 1, 0] = -1
    ids2 = ids.clone()
    ids2[int(indptr[1]) + int(sel[1, 0, 0])] = 10 ** 6
    o2, _, ws, _ = _attend(case, q, k, v, indptr, ids2, last, sel, ws=ws)
    assert pkx.workspace_status(ws) == pkx.PKX_EDEVICE and o2.isfinite().all()
    o3, lse3, ws, s = _attend(case, *args, ws=ws)  # and a clean call after it
    assert pkx.workspace_status(ws) == pkx.PKX_OK
    R.check_attention(o3, lse3, _reference(case, *args, *s))


def test_every_page_selected_is_plain_decode():
    """With every page selected, the call computes what decode attention over
    the expanded page table does."""
    case = dict(keys=[1000, 17, 640], page=32, hq=16, hkv=4, d=128, top=32, kv=torch.bfloat16, cap=0.0)
    q, k, v, indptr, ids, last, _ = (x.to(DEV) for x in _attend_case(case, 4))
    box = torch.zeros(k.shape[0] // 32, 4, 2, 128, dtype=torch.bfloat16, device=DEV)
    sel, _ = pkx.select_pages(q, box, indptr, ids, 32)
    o, o2 = torch.empty_like(q), torch.empty_like(q)
    lse, lse2 = (torch.empty(q.shape[:2], device=DEV) for _ in range(2))
    pkx.decode_attention_fwd_pages(q, o, k, v, indptr, ids, last, 32, sel, lse=lse)
    tptr, tidx = pkx.expand_paged_kv_indices(indptr, ids, last, 32, capacity=sum(case["keys"]))
    pkx.decode_attention_fwd(q, o2, k, v, tptr, tidx, lse=lse2)
    # two bf16 results of the same sums: half a step each, and P's rounding
    assert (o.float() - o2.float()).abs().max() <= 2.0 ** -6 * o2.float().abs().max()
    assert (lse - lse2).abs().max() <= 1e-4
