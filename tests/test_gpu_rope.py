"""GPU tests of the query / key norm with rotation and KV write."""
import pytest
import torch

import step_reference as R
from paged_kv_extend_gb300 import pkx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _table(n, r, g):
    angle = torch.rand(n, r // 2, generator=g, dtype=torch.float64) * 6.3
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _check(out, ref, size):
    """One rounding to bf16 (2^-8 of the value) and fp32 work: the sum of at
    most 256 squares (2^-16, halved by the root), rsqrt, products: 2^-16 of the
    elements that enter."""
    out = out.double().cpu()
    nan = ref.isnan()
    assert torch.equal(out.isnan(), nan)
    err = (out - ref).abs() - 2.0 ** -8 * ref.abs() - 2.0 ** -16 * size - 1e-30
    assert not (err[~nan] > 0).any()


CASES = [  # n, hq, hkv, d, rotary, norm, interleaved, axes
    (1, 1, 1, 64, 64, "qk", False, 1),
    (7, 8, 2, 128, 128, "qk", False, 1),
    (33, 5, 3, 128, 64, "", True, 3),
    (65, 28, 4, 128, 32, "q", False, 2),
    (130, 3, 1, 256, 256, "k", True, 1),
    (19, 6, 6, 80, 80, "qk", False, 1),
    (9, 2, 2, 8, 0, "qk", False, 1),
    (11, 4, 4, 40, 16, "qk", True, 1),
    (5, 7, 1, 192, 64, "qk", False, 3),
    (4099, 9, 3, 64, 32, "qk", False, 1),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_64_bits(case):
    n, hq, hkv, d, r, norm, leaved, axes = case
    g = torch.Generator().manual_seed(n * 131 + d)
    q = (torch.randn(n, hq, d, generator=g) * 3).bfloat16()
    k = (torch.randn(n, hkv, d, generator=g) * 0.01).bfloat16()
    qw = (1 + torch.randn(d, generator=g) * 0.3).bfloat16() if "q" in norm else None
    kw = (torch.randn(d, generator=g) * 0.3).bfloat16() if "k" in norm else None
    table = _table(50, r, g) if r else None
    pos = torch.randint(0, 50, (n,) if axes == 1 else (axes, n), generator=g) if r else None
    axis = torch.randint(0, axes, (r // 2,), generator=g).to(torch.uint8) if axes > 1 else None
    on = lambda t: None if t is None else t.to(DEV)
    qo, ko = pkx.qk_norm_rope(on(q), on(k), on(pos), on(table), q_weight=on(qw), k_weight=on(kw), eps=1e-5,
                              weight_offset=0.5, interleaved=leaved, pair_axis=on(axis))
    _check(qo, *R.rope(q, qw, 1e-5, 0.5, pos, table, leaved, axis))
    _check(ko, *R.rope(k, kw, 1e-5, 0.5, pos, table, leaved, axis))


@pytest.mark.parametrize("kv", [torch.bfloat16, torch.float8_e4m3fn, torch.float8_e5m2], ids=str)
@pytest.mark.parametrize("n", [3, 700])
def test_kv_write_is_the_separate_calls(n, kv):
    """In place on a packed projection, into a strided pool: the pool gets what
    set_kv_buffer (or its fp8 form) stores for the returned keys, bit for bit;
    other slots, and tokens with a slot outside the pool, write nothing."""
    g = torch.Generator().manual_seed(n)
    hq, hkv, d, slots = 6, 2, 128, n + 9
    qkv = torch.randn(n, (hq + 2 * hkv) * d, generator=g).bfloat16().to(DEV)
    q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], -1))
    loc = torch.randperm(slots, generator=g)[:n]
    loc[0], loc[1] = -1, slots
    loc = loc.to(DEV)
    table, pos = _table(64, 128, g).to(DEV), torch.randint(0, 64, (n,), generator=g).to(DEV)
    w = (1 + torch.randn(d, generator=g) * 0.1).bfloat16().to(DEV)

    def pools():
        both = torch.full((slots, 2, hkv, d), 0.75, device=DEV).to(kv)
        return both[:, 0], both[:, 1]

    kb, vb = pools()
    kb2, vb2 = pools()
    want_q, want_k = pkx.qk_norm_rope(q, k, pos, table, q_weight=w, k_weight=w)
    if kv == torch.bfloat16:
        pkx.set_kv_buffer(kb2, vb2, loc, want_k, v)
    else:
        pkx.set_kv_buffer_fp8(kb2, vb2, loc, want_k, v, 0.7, 0.3)
    qo, ko = pkx.qk_norm_rope(q, k, pos, table, q_out=q, k_out=k, q_weight=w, k_weight=w, cache_loc=loc, v=v,
                              k_buffer=kb, v_buffer=vb, k_scale=0.7, v_scale=0.3)
    assert qo.data_ptr() == q.data_ptr() and ko.data_ptr() == k.data_ptr()
    assert torch.equal(qo, want_q) and torch.equal(ko, want_k)
    raw = lambda t: t.contiguous().view(torch.uint8)
    assert torch.equal(raw(kb), raw(kb2)) and torch.equal(raw(vb), raw(vb2))


def test_keys_alone_and_no_rotation():
    n, d = 5, 64
    k = torch.randn(n, 2, d, device=DEV).bfloat16()
    kb = torch.zeros(8, 2, d, dtype=torch.bfloat16, device=DEV)
    loc = torch.arange(n, device=DEV) + 2
    q, ko = pkx.qk_norm_rope(k, k, cache_loc=loc, k_buffer=kb)
    assert torch.equal(q, k) and torch.equal(ko, k) and torch.equal(kb[2:7], k) and not kb[:2].any()
    e = torch.empty(0, 2, d, dtype=torch.bfloat16, device=DEV)
    q, ko = pkx.qk_norm_rope(e, e, cache_loc=loc[:0], v=e, k_buffer=kb, v_buffer=kb.clone())
    assert q.shape == e.shape


def test_positions_outside_the_table():
    """NaN in the rotated dims of the tokens at fault, the others untouched."""
    n, d, r = 6, 64, 32
    g = torch.Generator().manual_seed(1)
    q = torch.randn(n, 3, d, generator=g).bfloat16()
    pos = torch.tensor([0, -1, 9, 10, 2 ** 40, 3])
    table = _table(10, r, g)
    for leaved in (False, True):
        qo, ko = pkx.qk_norm_rope(q.to(DEV), q.to(DEV), pos.to(DEV), table.to(DEV), interleaved=leaved)
        _check(qo, *R.rope(q, None, 0, 0, pos, table, leaved, None))
        assert qo[[1, 3, 4], :, :r].isnan().all() and not qo[:, :, r:].isnan().any()
    axis = torch.full((r // 2,), 1, dtype=torch.uint8)
    axis[3] = 2  # no such axis
    two = torch.stack([torch.zeros(n, dtype=torch.int64), pos])
    qo, _ = pkx.qk_norm_rope(q.to(DEV), q.to(DEV), two.to(DEV), table.to(DEV), pair_axis=axis.to(DEV))
    _check(qo, *R.rope(q, None, 0, 0, two, table, False, axis))
    assert qo[:, :, 3].isnan().all() and qo[:, :, 19].isnan().all()


def test_nan_and_infinite_rows_stay_their_own():
    q = torch.randn(4, 2, 128, device=DEV).bfloat16()
    q[1, 0, 5] = float("nan")
    q[2, 1, 7] = float("inf")
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    qo, _ = pkx.qk_norm_rope(q, q, q_weight=w)
    assert qo[1, 0].isnan().all() and not qo[1, 1].isnan().any() and not qo[[0, 3]].isnan().any()
    zero, _ = pkx.qk_norm_rope(torch.zeros_like(q), q, q_weight=w, eps=0.0)
    assert zero.isnan().all()  # 0 / 0 by the formula
    zero, _ = pkx.qk_norm_rope(torch.zeros_like(q), q, q_weight=w)
    assert not zero.any()
