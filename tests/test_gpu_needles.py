"""Decode over selected pages and with shared prefixes reads every key once, at every
place where its work is cut: a few keys that outweigh all others for one query each
(needles) stand at both sides of every boundary, so that one left out or read twice
moves that query's lse by 1 / 80 at least (0.012 against a bound of 0.001) and its output by
|v| / 80.  The CPU test plants those mistakes in the reference."""
import random

import pytest
import torch

import step_reference as R
from paged_kv_extend_gb300 import pkx

DEV = "cuda:0"
BF, E4, E5 = torch.bfloat16, torch.float8_e4m3fn, torch.float8_e5m2
SCALE, LOGIT, MOST = 0.1, 30.0, 80


def _plant(q, k, ks, places, r):
    """places[b][h]: the pool slots that the queries of (sequence, KV head) read, in the
    order that is cut, and the ranks (into that list) of the keys to plant.  Sets the
    needles in ``k``; returns how many and the places that no query was left for."""
    hkv = k.shape[1]
    group = q.shape[1] // hkv
    taken, left = set(), []
    for b in range(q.shape[0]):
        for h in range(hkv):
            slots, ranks = places[b][h]
            want = [slots[i] for i in ranks if (slots[i], h) not in taken]
            r.shuffle(want)
            for g in range(group):
                row, want = want[:MOST], want[MOST:]
                x = q[b, h * group + g].float()
                needle = (x * (LOGIT / (SCALE * ks * float(x.square().sum())))).to(k.dtype)
                for s in row:
                    k[s, h] = needle
                taken |= {(s, h) for s in row}
            left += [(b, h, s) for s in want]
    return len(taken), [x for x in left if (x[2], x[1]) not in taken]


def _edges(n, *starts):
    """Ranks on both sides of the cuts into runs of 64 (and 128) from each start."""
    out = {0, n - 1}
    for s in starts:
        out |= {x for c in range(s, n + 64, 64) for x in (c - 1, c)}
    return sorted(x for x in out if 0 <= x < n)


def _attend(q, k, v, lists, scale=SCALE, ks=1.0, vs=1.0):
    """Reference over lists[b][h] of slots."""
    hkv = k.shape[1]
    g = q.shape[1] // hkv
    o, size = (torch.zeros(q.shape, dtype=torch.float64) for _ in range(2))
    lse = torch.zeros(q.shape[:2], dtype=torch.float64)
    k, v = k.double() * ks, v.double() * vs
    for b in range(q.shape[0]):
        for h in range(hkv):
            rows, at = slice(h * g, (h + 1) * g), torch.tensor(lists[b][h], dtype=torch.int64)
            o[b, rows], lse[b, rows], size[b, rows] = R.attend(q[b, rows].double(), k[at, h], v[at, h], scale)
    return o, lse, size


# ------------------------------------------------------------- shared prefixes
SHARED = [  # groups (shared keys, own keys of each member), alone, before, hq, hkv, d, kv
    ([(300, [5, 0, 70, 129])], [0, 40, 1], [], 12, 3, 64, BF),
    ([(1000, [9, 0, 130, 300, 1] * 13)], [0, 700], [], 32, 8, 128, BF),
    ([(3001, [5] * 18 + [0] * 19)], [], [33, 0], 28, 4, 128, BF),
    ([(2222, [64] * 12), (1999, [2] * 8)], [0, 900], [], 8, 8, 128, E4),
    ([(6100, [3] * 120)], [], [], 9, 1, 64, E5),
    ([(5000, [40] * 8)], [6], [], 64, 4, 128, BF),
    ([(6000, [100, 50])], [9000], [], 4, 1, 128, BF),           # read by each
    ([(700, [40, 0, 3, 900])], [6, 0], [2], 34, 2, 128, BF),    # 17 heads
    ([(900, [40, 0, 3])], [6, 0, 1500], [], 80, 2, 64, E4),     # 40 heads
]


def _shared_case(case, seed):
    groups, alone, before, hq, hkv, d, kv = case
    g, r = torch.Generator().manual_seed(seed), random.Random(seed)
    slots = sum(before) + sum(alone) + sum(s + sum(o) for s, o in groups) + 13
    free = torch.randperm(slots, generator=g).tolist()
    take = lambda n: [free.pop() for _ in range(n)]
    lists, starts = [], []
    for t in before:
        lists.append(take(t)), starts.append(0)
    for s, own in groups:
        prefix = take(s)
        for t in own:
            lists.append(prefix + take(t)), starts.append(s)
    for t in alone:
        lists.append(take(t)), starts.append(0)
    indptr = torch.tensor([0] + torch.tensor([len(x) for x in lists]).cumsum(0).tolist(), dtype=torch.int32)
    idx = torch.tensor([i for x in lists for i in x], dtype=torch.int32)
    first = len(before)
    gptr = torch.tensor([first] + (first + torch.tensor([len(o) for _, o in groups]).cumsum(0)).tolist(), dtype=torch.int32)
    shared = torch.tensor([s for s, _ in groups], dtype=torch.int32)
    k, v = (torch.randn(slots, hkv, d, generator=g).to(kv) for _ in range(2))
    q = torch.randn(len(lists), hq, d, generator=g).bfloat16()
    ks, vs = (1.0, 1.0) if kv == BF else (0.37, 1.9)
    places = [[(x, _edges(len(x), 0, s) if x else []) for _ in range(hkv)] for x, s in zip(lists, starts)]
    count, left = _plant(q, k, ks, places, r)
    assert not left, f"{len(left)} places without a query"
    return q, k, v, indptr, idx, gptr, shared, [[x] * hkv for x in lists], ks, vs, count


@pytest.mark.gpu
@pytest.mark.parametrize("case", SHARED, ids=lambda c: f"{[(s, len(o)) for s, o in c[0]]}-{c[3]}/{c[4]}x{c[5]}")
def test_shared_prefixes(case):
    q, k, v, indptr, idx, gptr, shared, lists, ks, vs, _ = _shared_case(case, 21)
    on = [x.to(DEV) for x in (q, k, v, indptr, idx, gptr, shared)]
    o, lse = torch.empty_like(on[0]), torch.empty(q.shape[:2], device=DEV)
    ws = pkx.decode_attention_fwd_shared(on[0], o, *on[1:], sm_scale=SCALE, lse=lse, k_scale=ks, v_scale=vs)
    assert pkx.workspace_status(ws) == pkx.PKX_OK
    R.check_attention(o, lse, _attend(q, k, v, lists, ks=ks, vs=vs))


# -------------------------------------------------------------- selected pages
PAGES = [  # keys of each sequence, page, hq, hkv, d, top, kv
    ([700, 0, 1, 129, 40], 16, 12, 3, 64, 9, BF),
    ([9000], 64, 4, 1, 128, 141, BF),
    ([4000, 31], 16, 16, 1, 128, 240, BF),
    ([3000, 9], 24, 9, 1, 64, 100, E4),
    ([900, 5, 64], 32, 28, 4, 128, 11, E5),
    ([5000], 200, 128, 1, 64, 25, BF),                          # more than 16 heads a KV head
    ([4000, 0, 90], 64, 34, 2, 128, 60, E4),
]


def _pages_case(case, seed):
    keys, page, hq, hkv, d, top, kv = case
    g, r = torch.Generator().manual_seed(seed), random.Random(seed)
    pages = [-(-t // page) for t in keys]
    indptr = torch.tensor([0] + torch.tensor(pages).cumsum(0).tolist(), dtype=torch.int32)
    ids = torch.randperm(sum(pages) + 3, generator=g)[:sum(pages)].to(torch.int32)
    last = torch.tensor([t - (p - 1) * page if p else 0 for t, p in zip(keys, pages)], dtype=torch.int32)
    k, v = (torch.randn((sum(pages) + 3) * page, hkv, d, generator=g).to(kv) for _ in range(2))
    q = torch.randn(len(keys), hq, d, generator=g).bfloat16()
    sel = torch.full((len(keys), hkv, top), -1, dtype=torch.int32)
    places = []
    for b, n in enumerate(pages):
        places.append([])
        for h in range(hkv):
            pick = sorted(r.sample(range(n), min(n, top)))
            sel[b, h, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
            slots, cut = [], set()
            for e, s in enumerate(pick):
                held = int(last[b]) if s == n - 1 else page
                start = int(ids[int(indptr[b]) + s]) * page
                # cuts by places (every page counts whole) and, below, by keys
                cut |= {len(slots) + x for x in (*(j for j in range(held) if (e * page + j) % 64 in (0, 63)), 0, held - 1)}
                slots += range(start, start + held)
            places[-1].append((slots, sorted(cut | set(_edges(len(slots), 0))) if slots else []))
    ks, vs = (1.0, 1.0) if kv == BF else (0.37, 1.9)
    count, left = _plant(q, k, ks, places, r)
    assert not left, f"{len(left)} places without a query"
    return q, k, v, indptr, ids, last, sel, [[s for s, _ in x] for x in places], ks, vs, count


@pytest.mark.gpu
@pytest.mark.parametrize("case", PAGES, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}/{c[3]}x{c[4]}")
def test_selected_pages(case):
    q, k, v, indptr, ids, last, sel, lists, ks, vs, _ = _pages_case(case, 22)
    on = [x.to(DEV) for x in (q, k, v, indptr, ids, last, sel)]
    o, lse = torch.empty_like(on[0]), torch.empty(q.shape[:2], device=DEV)
    ws = pkx.decode_attention_fwd_pages(on[0], o, *on[1:6], case[1], on[6], SCALE, lse=lse, k_scale=ks, v_scale=vs)
    assert pkx.workspace_status(ws) == pkx.PKX_OK
    R.check_attention(o, lse, _attend(q, k, v, lists, ks=ks, vs=vs))


# ------------------------------------------------------------- the test itself
@pytest.mark.parametrize("make,case", [(_shared_case, SHARED[0]), (_shared_case, SHARED[7]), (_pages_case, PAGES[0]),
                                       (_pages_case, PAGES[3])], ids=["shared", "17 heads", "pages", "fp8 pages"])
def test_a_needle_left_out_or_read_twice_is_seen(make, case):
    q, k, v, *_, lists, ks, vs, count = make(case, 23)
    o, lse, size = _attend(q, k, v, lists, ks=ks, vs=vs)
    R.check_attention(o.bfloat16(), lse.float(), (o, lse, size))
    r, tried = random.Random(1), 0
    start = 0 if make is _pages_case else len(case[2])
    hkv = k.shape[1]
    group = q.shape[1] // hkv
    for b in range(len(lists)):
        for h in range(hkv):
            rows, slots = slice(h * group, (h + 1) * group), lists[b][h]
            if not slots:
                continue
            logits = q[b, rows].double() @ (k[slots, h].double() * ks).T * SCALE
            at = [i for i in range(len(slots)) if float(logits[:, i].max()) > 0.8 * LOGIT]
            for i in r.sample(at, min(len(at), 24)):
                for wrong in (slots[:i] + slots[i + 1:], slots + [slots[i]]):
                    bad = [x.clone() for x in (o, lse)]
                    kk, vv = (x[wrong, h].double() * f for x, f in ((k, ks), (v, vs)))
                    bad[0][b, rows], bad[1][b, rows], _ = R.attend(q[b, rows].double(), kk, vv, SCALE)
                    with pytest.raises(AssertionError):
                        R.check_attention(bad[0].bfloat16(), bad[1].float(), (o, lse, size))
                    tried += 1
    assert tried >= 40 and count >= 40
