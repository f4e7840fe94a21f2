"""CPU tests of a decode step's operators: the reference against hand values,
and the refusals of the entry points (nothing reaches a GPU)."""
import math

import pytest
import torch

import step_reference as R
from paged_kv_extend_gb300 import build as pkx_build
from paged_kv_extend_gb300 import pkx


@pytest.fixture(scope="module")
def lib():
    pkx_build.build()
    return pkx.load_library()


# --------------------------------------------------------------- the reference
def test_reference_rotation():
    x = torch.tensor([[[3.0, 4.0, 1.0, 2.0]]]).bfloat16()
    quarter = torch.tensor([[0.0, 1.0, 1.0, 0.0]])  # pair 0 by a quarter turn, pair 1 not
    pos = torch.zeros(1, dtype=torch.int64)
    out, _ = R.rope(x, None, 0.0, 0.0, pos, quarter, False, None)
    assert out.flatten().tolist() == [-1.0, 4.0, 3.0, 2.0]  # pairs (3, 1) and (4, 2)
    out, _ = R.rope(x, None, 0.0, 0.0, pos, quarter, True, None)
    assert out.flatten().tolist() == [-4.0, 3.0, 1.0, 2.0]  # pairs (3, 4) and (1, 2)
    w = torch.tensor([1.0, 0.0, 2.0, -1.0]).bfloat16()
    out, _ = R.rope(x, w, 0.0, 1.0, None, None, False, None)
    rms = math.sqrt(30 / 4)
    assert torch.allclose(out.flatten(), torch.tensor([6.0, 4.0, 3.0, 0.0], dtype=torch.float64) / rms)


def test_reference_selection():
    """A box that holds one key scores that key's logit; wider boxes score more."""
    g = torch.Generator().manual_seed(1)
    keys = torch.randn(6, 64, generator=g).bfloat16()
    q = torch.randn(2, 64, generator=g).bfloat16()
    box = torch.stack([keys, keys], 1)
    want = (q.double() @ keys.double().T).sum(0)
    assert (R.scores(q, box).double() - want).abs().max() < 1e-4
    wide = torch.stack([keys - 1, keys + 1], 1)
    assert (R.scores(q, wide) > R.scores(q, box)).all()
    sel = R.select(q[None], box[:, None], torch.tensor([0, 6]), torch.arange(6), 3, 1, 1)
    middle = 1 + int(R.scores(q, box)[1:5].argmax())
    assert sel.flatten().tolist() == [0, middle, 5]


def test_reference_attention():
    q, k = torch.zeros(1, 2, dtype=torch.float64), torch.zeros(3, 2, dtype=torch.float64)
    v = torch.tensor([[1.0, -2.0], [2.0, 0.0], [6.0, 5.0]], dtype=torch.float64)
    o, lse, size = R.attend(q, k, v, 1.0)
    assert torch.allclose(o, v.mean(0, keepdim=True)) and abs(float(lse) - math.log(3)) < 1e-12
    assert torch.allclose(size, v.abs().mean(0, keepdim=True))


# -------------------------------------------------------------------- refusals
P = 0x10000  # an aligned address that no check dereferences
INVALID, UNSUPPORTED, WORKSPACE, OK = (pkx.PKX_EINVAL, pkx.PKX_EUNSUPPORTED, pkx.PKX_EWORKSPACE, pkx.PKX_OK)


def _rope(lib, **over):
    a = dict(q=P, qs=(1024, 128), k=P, ks=(256, 128), v=P, vs=(256, 128), n=4, hq=8, hkv=2, d=128, pos=P, axes=1,
             axis=None, table=P, rows=10, r=128, leaved=0, qw=P, kw=None, eps=1e-6, off=0.0, qo=P, qos=(1024, 128),
             ko=P, kos=(256, 128), loc=P, kb=P, kbs=(256, 128), vb=P, vbs=(256, 128), slots=9, fmt=0, s=1.0, t=1.0)
    a.update(over)
    return lib.pkx_qk_norm_rope(
        a["q"], *a["qs"], a["k"], *a["ks"], a["v"], *a["vs"], a["n"], a["hq"], a["hkv"], a["d"], a["pos"], a["axes"],
        a["axis"], a["table"], a["rows"], a["r"], a["leaved"], a["qw"], a["kw"], a["eps"], a["off"], a["qo"],
        *a["qos"], a["ko"], *a["kos"], a["loc"], a["kb"], *a["kbs"], a["vb"], *a["vbs"], a["slots"], a["fmt"], a["s"],
        a["t"], None)


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), INVALID), (dict(hq=0), INVALID), (dict(hkv=-1), INVALID), (dict(d=0), INVALID), (dict(d=100), INVALID),
    (dict(d=264), UNSUPPORTED), (dict(r=24), INVALID), (dict(r=144), INVALID), (dict(r=-16), INVALID),
    (dict(n=1 << 40), UNSUPPORTED), (dict(hq=(1 << 20) + 1), UNSUPPORTED), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(off=float("inf")), INVALID), (dict(pos=None), INVALID),
    (dict(pos=P + 4), INVALID), (dict(table=None), INVALID), (dict(table=P + 8), INVALID), (dict(rows=0), INVALID),
    (dict(axes=0), INVALID), (dict(axes=3), INVALID), (dict(q=None), INVALID), (dict(q=P + 8), INVALID),
    (dict(qs=(1024, 100)), INVALID), (dict(ks=(-8, 128)), INVALID), (dict(qo=None), INVALID), (dict(ko=P + 2), INVALID),
    (dict(qw=P + 8), INVALID), (dict(kw=P + 2), INVALID), (dict(loc=None), INVALID), (dict(loc=P + 4), INVALID),
    (dict(kb=None), INVALID), (dict(vb=None), INVALID), (dict(vs=(256, 4)), INVALID), (dict(kbs=(256, 4)), INVALID),
    (dict(slots=-1), INVALID), (dict(fmt=9), INVALID), (dict(fmt=1, s=0.0), INVALID),
    (dict(fmt=2, t=float("inf")), INVALID),
], ids=str)
def test_rope_refuses(lib, over, code):
    assert _rope(lib, **over) == code and lib.pkx_last_error_string()


def test_rope_of_nothing(lib):
    assert _rope(lib, n=0, q=None, k=None, v=None, pos=None, loc=None) == OK


def _bounds(lib, **over):
    a = dict(k=P, ks=(1024, 128), fmt=0, page=16, pages=8, hkv=8, d=128, ids=P, lens=None, n=4, out=P)
    a.update(over)
    return lib.pkx_update_page_bounds(a["k"], *a["ks"], a["fmt"], a["page"], a["pages"], a["hkv"], a["d"], a["ids"],
                                      a["lens"], a["n"], a["out"], None)


@pytest.mark.parametrize("over,code", [
    (dict(fmt=3), INVALID), (dict(page=0), INVALID), (dict(pages=-1), INVALID), (dict(n=-1), INVALID),
    (dict(hkv=0), INVALID), (dict(d=12), INVALID), (dict(d=2048), UNSUPPORTED), (dict(k=None), INVALID),
    (dict(ks=(1024, 4)), INVALID), (dict(out=None), INVALID), (dict(out=P + 8), INVALID), (dict(ids=None), INVALID),
    (dict(ids=P + 2), INVALID), (dict(lens=P + 1), INVALID), (dict(n=1 << 33), UNSUPPORTED),
], ids=str)
def test_bounds_refuse(lib, over, code):
    assert _bounds(lib, **over) == code and lib.pkx_last_error_string()


def test_bounds_of_nothing(lib):
    assert _bounds(lib, n=0, k=None, out=None, ids=None) == OK


def _select(lib, **over):
    a = dict(q=P, box=P, pages=8, ptr=P, idx=P, n=40, batch=2, hq=8, hkv=2, d=128, top=4, first=1, last=1, out=P, ws=P,
             wsb=1 << 40)
    a.update(over)
    return lib.pkx_select_pages(a["q"], a["box"], a["pages"], a["ptr"], a["idx"], a["n"], a["batch"], a["hq"], a["hkv"],
                                a["d"], a["top"], a["first"], a["last"], a["out"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), INVALID), (dict(hq=7), INVALID), (dict(hq=258), UNSUPPORTED), (dict(d=96), UNSUPPORTED),
    (dict(d=576), UNSUPPORTED), (dict(top=0), INVALID), (dict(top=4097), UNSUPPORTED), (dict(first=-1), INVALID),
    (dict(first=3, last=2), INVALID), (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), INVALID), (dict(pages=-1), INVALID),
    (dict(n=-1), INVALID), (dict(n=1 << 31), UNSUPPORTED), (dict(q=None), INVALID), (dict(box=None), INVALID),
    (dict(box=P + 8), INVALID), (dict(ptr=None), INVALID), (dict(idx=None), INVALID), (dict(idx=P + 2), INVALID),
    (dict(out=None), INVALID), (dict(out=P + 2), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=300), WORKSPACE),
    (dict(ws=P + 16), INVALID),
], ids=str)
def test_select_refuses(lib, over, code):
    assert _select(lib, **over) == code and lib.pkx_last_error_string()


def _pages(lib, **over):
    a = dict(q=P, o=P, k=P, v=P, ptr=P, idx=P, n=40, last=P, page=16, sel=P, top=4, batch=2, hq=8, hkv=2, lq=128,
             lv=128, st=(256, 128, 256, 128), slots=640, scale=0.0, cap=0.0, fmt=0, s=1.0, t=1.0, lse=None, ws=P,
             wsb=1 << 40)
    a.update(over)
    return lib.pkx_decode_attention_fwd_pages(
        a["q"], a["o"], a["k"], a["v"], a["ptr"], a["idx"], a["n"], a["last"], a["page"], a["sel"], a["top"],
        a["batch"], a["hq"], a["hkv"], a["lq"], a["lv"], *a["st"], a["slots"], a["scale"], a["cap"], a["fmt"], a["s"],
        a["t"], a["lse"], a["ws"], a["wsb"], None)


def _shared(lib, **over):
    a = dict(q=P, o=P, k=P, v=P, ptr=P, idx=P, n=640, gptr=P, lens=P, groups=1, batch=2, hq=8, hkv=2, lq=128, lv=128,
             st=(256, 128, 256, 128), slots=640, scale=0.0, cap=0.0, fmt=0, s=1.0, t=1.0, lse=None, ws=P, wsb=1 << 40)
    a.update(over)
    return lib.pkx_decode_attention_fwd_shared(
        a["q"], a["o"], a["k"], a["v"], a["ptr"], a["idx"], a["n"], a["gptr"], a["lens"], a["groups"], a["batch"], a["hq"],
        a["hkv"], a["lq"], a["lv"], *a["st"], a["slots"], a["scale"], a["cap"], a["fmt"], a["s"], a["t"], a["lse"],
        a["ws"], a["wsb"], None)


BOTH = [
    (dict(batch=-1), INVALID), (dict(hq=7), INVALID), (dict(hq=258), UNSUPPORTED), (dict(lq=576, lv=512), UNSUPPORTED),
    (dict(lq=192, lv=128), UNSUPPORTED), (dict(lq=64, lv=128), UNSUPPORTED), (dict(scale=float("nan")), INVALID),
    (dict(cap=float("inf")), INVALID), (dict(fmt=3), INVALID), (dict(fmt=1, s=-1.0), INVALID), (dict(q=None), INVALID),
    (dict(o=P + 8), INVALID), (dict(k=None), INVALID), (dict(v=P + 4), INVALID), (dict(st=(256, 100, 256, 128)), INVALID),
    (dict(st=(256, 128, -8, 128)), INVALID), (dict(ptr=None), INVALID), (dict(idx=P + 1), INVALID),
    (dict(lse=P + 2), INVALID), (dict(slots=0), INVALID), (dict(slots=1 << 31), UNSUPPORTED),
    (dict(fmt=1, st=(264, 128, 256, 128)), INVALID), (dict(fmt=2, st=(256, 128, 256, 136)), INVALID),
]


@pytest.mark.parametrize("over,code", BOTH + [
    (dict(top=0), INVALID), (dict(top=5000), UNSUPPORTED), (dict(page=0), INVALID), (dict(n=-1), INVALID),
    (dict(idx=None), INVALID), (dict(last=None), INVALID), (dict(sel=P + 2), INVALID),
    (dict(page=1 << 28, top=8), UNSUPPORTED),
], ids=str)
def test_pages_refuse(lib, over, code):
    assert _pages(lib, **over) == code and lib.pkx_last_error_string()


@pytest.mark.parametrize("over,code", BOTH + [
    (dict(groups=-1), INVALID), (dict(n=-1), INVALID), (dict(idx=None), INVALID), (dict(gptr=None), INVALID), (dict(lens=P + 2), INVALID),
], ids=str)
def test_shared_refuse(lib, over, code):
    assert _shared(lib, **over) == code and lib.pkx_last_error_string()


def test_decode_of_nothing(lib):
    assert _pages(lib, batch=0, q=None, k=None, ws=None) == OK
    assert _shared(lib, batch=0, q=None, k=None, ws=None) == OK
    assert _select(lib, batch=0, q=None, ws=None) == OK


def test_workspace_sizes():
    assert pkx.select_pages_workspace_size(-1, 1, 5) == 0 and pkx.select_pages_workspace_size(2, 0, 5) == 0
    assert pkx.select_pages_workspace_size(4, 8, 1000) >= 4 * 8 * 1000
    bad = [(-1, 8, 2, 64, 64), (1, 7, 2, 64, 64), (1, 8, 2, 96, 96), (1, 8, 2, 64, 128), (1, 258, 2, 64, 64)]
    for shape in bad:
        assert pkx.decode_pages_workspace_size(*shape, 16, 4) == 0
        assert pkx.decode_shared_workspace_size(shape[0], 1, *shape[1:]) == 0
    assert pkx.decode_pages_workspace_size(1, 8, 2, 64, 64, 0, 4) == 0
    assert pkx.decode_pages_workspace_size(1, 8, 2, 64, 64, 16, 5000) == 0
    assert pkx.decode_shared_workspace_size(1, -1, 8, 2, 64, 64) == 0
    small, large = (pkx.decode_shared_workspace_size(b, b // 2, 32, 8, 128, 128) for b in (4, 400))
    assert 0 < small < large


def test_binding_refuses_host_tensors_and_shapes():
    bf, i32 = torch.bfloat16, torch.int32
    x, k = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(16, 2, 64, dtype=bf)
    ptr, idx = torch.zeros(4, dtype=i32), torch.zeros(2, dtype=i32)
    calls = [lambda: pkx.qk_norm_rope(x, x), lambda: pkx.update_page_bounds(k, torch.zeros(1, 2, 2, 64, dtype=bf), idx, 16),
             lambda: pkx.select_pages(x, torch.zeros(1, 2, 2, 64, dtype=bf), ptr, idx, 2),
             lambda: pkx.decode_attention_fwd_pages(x, x, k, k, ptr, idx, ptr[:3], 16, torch.zeros(3, 2, 2, dtype=i32)),
             lambda: pkx.decode_attention_fwd_shared(x, x, k, k, ptr, idx, idx, idx[:1])]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call()
