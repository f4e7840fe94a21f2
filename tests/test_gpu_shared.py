"""GPU tests of decode attention for sequences in groups that share a prefix."""
import pytest
import torch

import step_reference as R
from paged_kv_extend_gb300 import pkx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _case(groups, alone, before, hq, hkv, d, kv, seed):
    """groups: (shared, own keys of each member); alone / before: keys of the
    sequences behind and in front of the groups."""
    g = torch.Generator().manual_seed(seed)
    lens, lists = [], []
    total = sum(before) + sum(alone) + sum(s + sum(o) for s, o in groups)
    slots = total + 13
    free = torch.randperm(slots, generator=g).tolist()
    take = lambda n: [free.pop() for _ in range(n)]
    for t in before:
        lists.append(take(t))
    for s, own in groups:
        pre = take(s)
        lists += [pre + take(t) for t in own]
    for t in alone:
        lists.append(take(t))
    lens = [len(x) for x in lists]
    indptr = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)
    idx = torch.tensor([i for x in lists for i in x], dtype=torch.int32)
    gptr = torch.tensor([len(before)] + (len(before) + torch.tensor([len(o) for _, o in groups]).cumsum(0)).tolist()
                        if groups else [len(before)], dtype=torch.int32)
    shared = torch.tensor([s for s, _ in groups], dtype=torch.int32)
    k, v = (torch.randn(slots, hkv, d, generator=g).to(kv) for _ in range(2))
    q = torch.randn(len(lens), hq, d, generator=g).bfloat16()
    return q, k, v, indptr, idx, gptr, shared


def _run(args, scale=0.1, cap=0.0, ks=1.0, vs=1.0, ws=None):
    q, *rest = (x.to(DEV) for x in args)
    o, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device=DEV)
    ws = pkx.decode_attention_fwd_shared(q, o, *rest, sm_scale=scale, logit_cap=cap, lse=lse, k_scale=ks, v_scale=vs,
                                         workspace=ws)
    return o, lse, ws


def _reference(args, scale=0.1, cap=0.0, ks=1.0, vs=1.0):
    q, k, v, indptr, idx, _, _ = args
    hkv = k.shape[1]
    g = q.shape[1] // hkv
    o, size = (torch.zeros(q.shape, dtype=torch.float64) for _ in range(2))
    lse = torch.zeros(q.shape[:2], dtype=torch.float64)
    k, v = k.double() * ks, v.double() * vs
    for b in range(q.shape[0]):
        at = idx[int(indptr[b]):int(indptr[b + 1])].long()
        for h in range(hkv):
            rows = slice(h * g, (h + 1) * g)
            o[b, rows], lse[b, rows], size[b, rows] = R.attend(q[b, rows].double(), k[at, h], v[at, h], scale, cap)
    return o, lse, size


BF, E4, E5 = torch.bfloat16, torch.float8_e4m3fn, torch.float8_e5m2
CASES = [  # groups, alone, before, hq, hkv, d, kv, cap
    ([(128, [0, 0])], [], [], 1, 1, 64, BF, 0.0),
    ([(300, [5, 0, 70, 129])], [0, 40, 1], [], 12, 3, 64, BF, 0.0),
    ([(1000, [3] * 33), (129, [200, 0]), (50, [1, 2, 3])], [7], [90, 0], 32, 8, 128, BF, 0.0),
    ([(513, [10] * 65)], [], [], 32, 8, 128, BF, 0.0),          # blocks of 64 and 1 sequence
    ([(700, [4, 5] * 18 + [6])], [300], [], 28, 4, 128, BF, 3.0),  # 18 sequences a tile, 37
    ([(257, [9, 0, 3]), (0, [5, 5]), (200, [8])], [], [], 128, 1, 128, BF, 0.0),  # a token a tile
    ([(400, [20, 30, 1]), (1, [2, 2])], [0], [3], 8, 2, 128, E4, 0.0),
    ([(260, [0, 500, 3])], [64], [], 8, 1, 64, E5, 0.0),
    ([], [5, 0, 300], [], 8, 2, 64, BF, 0.0),
    ([(6000, [100, 50])], [9000], [], 4, 1, 128, BF, 0.0),
    ([(150, [1, 2])] * 40, [], [], 4, 2, 64, BF, 0.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{[(s, len(o)) for s, o in c[0]][:3]}-{c[3]}/{c[4]}x{c[5]}")
def test_against_64_bits(case):
    groups, alone, before, hq, hkv, d, kv, cap = case
    args = _case(groups, alone, before, hq, hkv, d, kv, 11)
    kw = dict(cap=cap) if kv == BF else dict(cap=cap, ks=0.37, vs=1.9)
    o, lse, ws = _run(args, **kw)
    assert pkx.workspace_status(ws) == pkx.PKX_OK
    R.check_attention(o, lse, _reference(args, **kw), cap)


# Sharing runs where it saves more than 88 << 20 elements of K and V, of groups of
# at most 16 query heads; all of these but the third do (it saves 82 << 20).
# Groups of more heads always share.
LARGE = [  # groups, alone, before, hq, hkv, d, kv, cap
    ([(1000, [9, 0, 130, 300, 1] * 13)], [0, 700], [], 32, 8, 128, BF, 0.0),   # blocks of 64 and 1 sequence
    ([(3001, [5] * 18 + [0] * 19)], [], [33, 0], 28, 4, 128, BF, 3.0),         # 18 sequences a tile, 37
    ([(2500, [4, 300, 0]), (129, [7, 7]), (2000, [1] * 9), (20, [3, 4])], [70], [5], 16, 16, 128, BF, 0.0),
    ([(2500, [4, 300, 0]), (129, [7, 7]), (4000, [1] * 9), (20, [3, 4])], [70], [5], 16, 16, 128, BF, 0.0),
    ([(2222, [64] * 12), (1999, [2] * 8)], [0, 900], [], 8, 8, 128, E4, 0.0),
    ([(6100, [3] * 120)], [], [], 9, 1, 64, E5, 0.0),                          # 14 sequences a tile
    ([(5000, [40] * 8)], [6], [], 64, 4, 128, BF, 0.0),                        # 16 heads
    ([(700, [40, 0, 3, 900])], [6, 0], [2], 34, 2, 128, BF, 0.0),              # 17 heads
    ([(900, [40, 0, 3])], [6, 0, 1500], [], 80, 2, 64, E4, 0.0),               # 40 heads
]


@pytest.mark.parametrize("case", LARGE, ids=lambda c: f"{[(s, len(o)) for s, o in c[0]][:3]}-{c[3]}/{c[4]}x{c[5]}")
def test_large_groups_against_64_bits(case):
    groups, alone, before, hq, hkv, d, kv, cap = case
    args = _case(groups, alone, before, hq, hkv, d, kv, 12)
    kw = dict(cap=cap) if kv == BF else dict(cap=cap, ks=0.37, vs=1.9)
    o, lse, ws = _run(args, **kw)
    assert pkx.workspace_status(ws) == pkx.PKX_OK
    saved = sum((len(o) - 1) * s for s, o in groups if s >= 128) * 2 * d * hkv
    shares = saved >= 88 << 20 or hq // hkv > 16
    assert (int(ws.view(torch.int32)[1]) > 0) == shares  # units of prefixes
    R.check_attention(o, lse, _reference(args, **kw), cap)


@pytest.mark.parametrize("keys,members,hq,hkv", [(200, 2, 32, 8), (3000, 17, 32, 8), (50, 3, 8, 2), (50, 3, 34, 2)])
def test_the_first_sequence_lists_the_prefix(keys, members, hq, hkv):
    """The others' entries below the shared length are not read, whether the
    prefix is shared or (few members) read by each."""
    args = _case([(keys, [9, 30] + [1] * (members - 2))], [], [], hq, hkv, 128, BF, 2)
    q, k, v, indptr, idx, gptr, shared = args
    want = _run(args)[:2]
    idx = idx.clone()
    for b in range(1, members):
        idx[int(indptr[b]):int(indptr[b]) + keys] = -1
    o, lse, ws = _run((q, k, v, indptr, idx, gptr, shared))
    assert pkx.workspace_status(ws) == pkx.PKX_OK
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("hq", [1, 17])
def test_many_sequences_and_groups(hq):
    """5000 sequences in 1500 groups: more than the scheduler's threads, and
    than its shared memory holds."""
    args = _case([(130 + i % 3, [i % 5, 2, 0]) for i in range(1500)], [i % 7 for i in range(500)], [], hq, 1, 64, BF, 3)
    o, lse, ws = _run(args)
    assert pkx.workspace_status(ws) == pkx.PKX_OK
    R.check_attention(o, lse, _reference(args))


def test_shared_lengths_past_a_sequence():
    """A group shares at most its shortest sequence's keys."""
    q, k, v, indptr, idx, gptr, _ = args = _case([(300, [9, 0, 100])], [20], [], 8, 2, 64, BF, 4)
    for s in (300, 10 ** 6):
        run = (q, k, v, indptr, idx, gptr, torch.tensor([s], dtype=torch.int32))
        o, lse, ws = _run(run)
        assert pkx.workspace_status(ws) == pkx.PKX_OK
        R.check_attention(o, lse, _reference(args))
    # a padded sequence of no keys in the group: nothing is shared
    indptr2 = torch.cat([indptr[:3], indptr[2:3], indptr[4:]])
    run = (q, k, v, indptr2, idx, gptr, torch.tensor([300], dtype=torch.int32))
    o, lse, ws = _run(run)
    ref = list(_reference(run))
    R.check_attention(o, lse, ref)
    assert not o[2].any()


def test_bad_groups_share_nothing_and_are_reported():
    q, k, v, indptr, idx, gptr, shared = args = _case([(200, [9, 30]), (150, [1, 2])], [], [], 4, 2, 64, BF, 6)
    ref = _reference(args)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    ws = None
    for gp, sh in ((i32(0, 3, 2), shared), (i32(0, 2, 5), shared), (i32(-1, 2, 4), shared), (gptr, i32(200, -1))):
        o, lse, ws = _run((q, k, v, indptr, idx, gp, sh), ws=ws)
        assert pkx.workspace_status(ws) == pkx.PKX_EDEVICE
        R.check_attention(o, lse, ref)
    o, lse, ws = _run(args, ws=ws)
    assert pkx.workspace_status(ws) == pkx.PKX_OK
    R.check_attention(o, lse, ref)
    # an indptr that decreases, or that passes the list: no keys, reported
    for at, value in ((2, int(indptr[1]) - 1), (4, int(indptr[4]) + 1), (1, -5)):
        broken = indptr.clone()
        broken[at] = value
        o, lse, ws = _run((q, k, v, broken, idx, gptr, shared), ws=ws)
        assert pkx.workspace_status(ws) == pkx.PKX_EDEVICE
        assert not o[at - 1].any() and (lse[at - 1] == float("-inf")).all() and o.isfinite().all()
    idx = idx.clone()
    idx[5] = k.shape[0]
    o, lse, ws = _run((q, k, v, indptr, idx, gptr, shared), ws=ws)
    assert pkx.workspace_status(ws) == pkx.PKX_EDEVICE and o.isfinite().all()


@pytest.mark.parametrize("keys,members,hkv", [(256, 3, 2), (9000, 20, 4)])
def test_nan_rows_stay_their_own(keys, members, hkv):
    """A NaN query is its own row's; a NaN key or value of the prefix reaches
    the whole group of its KV head and nobody else."""
    args = _case([(keys, [4, 5, 6] + [1] * (members - 3))], [40], [], 4 * hkv, hkv, 64, BF, 9)
    q, k, v, indptr, idx, gptr, shared = args
    q[1, 2, 3] = float("nan")
    o, lse, _ = _run(args)
    bad = torch.zeros(members + 1, 4 * hkv, dtype=torch.bool)
    bad[1, 2] = True
    assert torch.equal(o.isnan().any(-1).cpu(), bad) and torch.equal(lse.isnan().cpu(), bad)
    q[1, 2, 3] = 0.0
    k[int(idx[100]), 1, 0] = float("nan")
    o, lse, _ = _run(args)
    bad[:] = False
    bad[:members, 4:8] = True
    assert torch.equal(o.isnan().all(-1).cpu(), bad) and torch.equal(lse.isnan().cpu(), bad)


def test_infinite_logits_of_one_part():
    """A prefix whose keys outweigh all others, and one that vanishes."""
    args = _case([(256, [64, 3])], [], [], 4, 1, 64, BF, 10)
    for f in (30.0, 0.01):
        k = args[1].clone()
        k[args[4][:256].long()] *= f
        run = (args[0], k, *args[2:])
        o, lse, _ = _run(run, scale=1.0)
        ref = _reference(run, scale=1.0)
        # (logits of up to a few hundred: fp32 leaves 2^-24 * 300 * 64 terms)
        o, lse = o.double().cpu(), lse.double().cpu()
        assert ((o - ref[0]).abs() <= 2.0 ** -8 * ref[0].abs() + (2.0 ** -8 + 2.0 ** -9) * ref[2]).all()
        assert ((lse - ref[1]).abs() <= 1e-5 * ref[1].abs() + 1e-3).all()
