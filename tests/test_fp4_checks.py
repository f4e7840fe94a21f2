"""CPU tests of the 4-bit pool: the reference implementation against hand
values, and the refusals of the entry points (nothing reaches a GPU)."""
import pytest
import torch

import fp4_reference as R
from paged_kv_extend_gb300 import build as pkx_build
from paged_kv_extend_gb300 import pkx


@pytest.fixture(scope="module")
def lib():
    pkx_build.build()
    return pkx.load_library()


def test_reference_values():
    # 6.0 sets the scale to 1; the other elements are codes themselves
    row = [6.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, -6.0, -0.5, 0.25, 0.75, 2.5, 5.0, 0.26, -5.1, 0.0]
    codes, bscale = R.pack(torch.tensor([[row]]).bfloat16(), 1.0)
    assert bscale.flatten().tolist() == [0x38]  # e4m3 1.0
    nib = [n for b in codes.flatten().tolist() for n in (b & 15, b >> 4)]
    assert nib == [7, 1, 2, 3, 4, 5, 6, 15, 9, 0, 2, 4, 6, 1, 15, 0]
    assert R.unpack(codes, bscale).flatten().tolist()[:8] == row[:8]
    assert R.E4M3[0x7E] == 448.0 and R.E4M3[1] == 2.0 ** -9
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    assert t.tolist() == R.E4M3.tolist()


def test_reference_attention_matches_the_oracle():
    """The reference against the oracle where both are defined (window, cap)."""
    import oracle
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(50, 2, 64, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(1, 4, 64, generator=g).bfloat16()
    idx = torch.randperm(50, generator=g).to(torch.int32)
    for cap, window in ((0.0, -1), (3.0, 7)):
        ro, rl = oracle.decode_attention(q, k, v, torch.tensor([0, 50]), idx, 0.1, cap, window)
        at = idx.long()
        o, lse, _, _ = R.attend(q.double(), k[at].double(), v[at].double(),
                                R.visible(torch.tensor([49]), 50, window, 0), 0.1, cap)
        assert (o - ro).abs().max() < 1e-12 and (lse - rl).abs().max() < 1e-12


P = 0x10000  # an aligned address that no check dereferences


def _write(lib, **over):
    a = dict(k=P, kst=(1024, 128), v=P, vst=(1024, 128), loc=P, n=4, hkv=8, lk=128, lv=128, ks=1.0, vs=1.0,
             kc=P, kcs=(512, 64), kb=P, kbs=(64, 8), vc=P, vcs=(512, 64), vb=P, vbs=(64, 8), slots=16)
    a.update(over)
    return lib.pkx_set_kv_buffer_fp4(a["k"], *a["kst"], a["v"], *a["vst"], a["loc"], a["n"], a["hkv"], a["lk"],
                                     a["lv"], a["ks"], a["vs"], a["kc"], *a["kcs"], a["kb"], *a["kbs"],
                                     a["vc"], *a["vcs"], a["vb"], *a["vbs"], a["slots"], None)


def _read(lib, **over):
    a = dict(k=P, kst=(1024, 128), v=P, vst=(1024, 128), idx=P, n=4, hkv=8, lk=128, lv=128, ks=1.0, vs=1.0,
             kc=P, kcs=(512, 64), kb=P, kbs=(64, 8), vc=P, vcs=(512, 64), vb=P, vbs=(64, 8), slots=16)
    a.update(over)
    return lib.pkx_get_kv_buffer_fp4(a["kc"], *a["kcs"], a["kb"], *a["kbs"], a["vc"], *a["vcs"], a["vb"],
                                     *a["vbs"], a["slots"], a["idx"], a["n"], a["hkv"], a["lk"], a["lv"],
                                     a["ks"], a["vs"], a["k"], *a["kst"], a["v"], *a["vst"], None)


BAD_ROWS = [dict(ks=0.0), dict(vs=float("inf")), dict(ks=float("nan")), dict(n=-1), dict(hkv=0), dict(lk=24),
            dict(lv=8), dict(slots=-1), dict(k=None), dict(k=P + 8), dict(kst=(1024, 4)), dict(kc=None),
            dict(kc=P + 4), dict(kcs=(512, 12)), dict(kcs=(-8, 64)), dict(kb=None), dict(vb=None),
            dict(vc=P + 1), dict(vbs=(-1, 8))]


@pytest.mark.parametrize("over", BAD_ROWS, ids=str)
def test_write_and_read_refuse(lib, over):
    assert _write(lib, **over) == pkx.PKX_EINVAL and lib.pkx_last_error_string()
    assert _read(lib, **over) == pkx.PKX_EINVAL


def test_write_and_read_refuse_more(lib):
    assert _write(lib, loc=None) == pkx.PKX_EINVAL and _write(lib, loc=P + 4) == pkx.PKX_EINVAL
    assert _read(lib, idx=None) == pkx.PKX_EINVAL and _read(lib, idx=P + 2) == pkx.PKX_EINVAL
    assert _write(lib, n=1 << 40) == pkx.PKX_EUNSUPPORTED
    assert _read(lib, n=1 << 40) == pkx.PKX_EUNSUPPORTED
    assert _write(lib, n=0, k=None, kc=None, loc=None) == pkx.PKX_OK
    assert _read(lib, n=0, k=None, kc=None, idx=None) == pkx.PKX_OK


def _decode(lib, **over):
    a = dict(q=P, o=P, kc=P, kb=P, vc=P, vb=P, ptr=P, idx=P, batch=2, hq=8, hkv=2, lq=128, lv=128,
             st=(128, 64, 16, 8, 128, 64, 16, 8), slots=16, scale=0.0, cap=0.0, win=-1, first=0, ks=1.0, vs=1.0,
             lse=None, ws=P, wsb=1 << 40)
    a.update(over)
    return lib.pkx_decode_attention_fwd_fp4(
        a["q"], a["o"], a["kc"], a["kb"], a["vc"], a["vb"], a["ptr"], a["idx"], a["batch"], a["hq"], a["hkv"],
        a["lq"], a["lv"], *a["st"], a["slots"], a["scale"], a["cap"], a["win"], a["first"], a["ks"], a["vs"],
        a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), pkx.PKX_EINVAL), (dict(hq=6, hkv=4), pkx.PKX_EINVAL),
    (dict(hq=258, hkv=2), pkx.PKX_EUNSUPPORTED), (dict(lq=576, lv=512), pkx.PKX_EUNSUPPORTED),
    (dict(lq=192, lv=128), pkx.PKX_EUNSUPPORTED), (dict(lq=96, lv=96), pkx.PKX_EUNSUPPORTED),
    (dict(ks=-1.0), pkx.PKX_EINVAL), (dict(scale=float("nan")), pkx.PKX_EINVAL),
    (dict(ks=2.0 ** -65), pkx.PKX_EUNSUPPORTED), (dict(vs=2.0 ** 65), pkx.PKX_EUNSUPPORTED),
    (dict(first=-1), pkx.PKX_EINVAL), (dict(q=None), pkx.PKX_EINVAL), (dict(o=P + 8), pkx.PKX_EINVAL),
    (dict(kc=P + 8), pkx.PKX_EINVAL), (dict(kb=P + 4), pkx.PKX_EINVAL), (dict(vc=None), pkx.PKX_EINVAL),
    (dict(st=(128, 72, 16, 8, 128, 64, 16, 8)), pkx.PKX_EINVAL),
    (dict(st=(128, 64, 16, 4, 128, 64, 16, 8)), pkx.PKX_EINVAL),
    (dict(st=(1 << 31, 64, 16, 8, 128, 64, 16, 8)), pkx.PKX_EUNSUPPORTED),
    (dict(slots=0), pkx.PKX_EINVAL), (dict(slots=1 << 31), pkx.PKX_EUNSUPPORTED),
    (dict(ptr=None), pkx.PKX_EINVAL), (dict(idx=P + 2), pkx.PKX_EINVAL), (dict(lse=P + 2), pkx.PKX_EINVAL),
    (dict(ws=None), pkx.PKX_EWORKSPACE), (dict(wsb=100), pkx.PKX_EWORKSPACE), (dict(ws=P + 16), pkx.PKX_EINVAL),
], ids=str)
def test_decode_refuses(lib, over, code):
    assert _decode(lib, **over) == code and lib.pkx_last_error_string()


def test_decode_of_nothing(lib):
    assert _decode(lib, batch=0, q=None, kc=None, ws=None) == pkx.PKX_OK
    assert pkx.decode_fp4_workspace_size(1, 8, 2, 96, 96) == 0
    assert pkx.decode_fp4_workspace_size(1, 7, 2, 64, 64) == 0


def test_binding_refuses():
    """Host tensors, wrong types and shapes stop in the binding."""
    kc, kb = torch.zeros(4, 2, 32, dtype=torch.uint8), torch.zeros(4, 2, 4, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        pkx._fp4_half(kc, kb, "k_buffer")  # host tensors
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pkx.set_kv_buffer_fp4(kc, kb, kc, kb, torch.zeros(3, dtype=torch.int64), x, x)
    with pytest.raises(ValueError):
        pkx.get_kv_buffer_fp4(kc, kb, kc, kb, torch.zeros(3, dtype=torch.int32))
    ptr = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkx.decode_attention_fwd_fp4(x, x, kc, kb, kc, kb, ptr, ptr)


def test_windows_past_the_int_range():
    assert pkx._c_int(2 ** 32 + 5) == 2 ** 31 - 1 and pkx._c_int(-2 ** 40) == -2 ** 31 and pkx._c_int(7) == 7
