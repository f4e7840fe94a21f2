"""GPU tests of rows whose softmax sum is NaN: a NaN query, or a NaN key that
the row sees.  Such a row is NaN in o and in lse, in every form and however
its keys are split; it is not taken for a row without keys (o = 0, lse =
-inf), and every other row keeps its bits."""
import pytest
import torch

from gpu_cases import DEV, DeviceWorkload
from paged_kv_extend_gb300 import pkx
from paged_kv_extend_gb300 import workloads as W
from test_gpu_fp4_extend import Case
from test_gpu_streaming import Extend

pytestmark = pytest.mark.gpu
NAN = float("nan")

# (prefix, extend): one tile; a few tiles; many sequences (no row is split);
# few tokens on a long prefix (split keys, two streams); long and short ones
LENGTHS = [([0], [1]), ([100, 0, 300], [20, 5, 3]), ([150] * 160, [2] * 160), ([8000], [3]),
           ([6000, 10, 0], [70, 300, 2])]
DECODE_LENGTHS = [[1], [20, 100], [5000], [300, 0, 9000, 128, 129]]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkx.load_library()


def _check(got, clean, hit):
    """hit [rows, hq]: the rows that see a NaN."""
    hit = hit.to(DEV)
    (o, lse), (co, cl) = got, clean
    assert not torch.isnan(co).any() and not torch.isnan(cl).any()
    assert torch.isnan(o[hit]).all(), "an output row that sees a NaN is not NaN"
    assert torch.isnan(lse[hit]).all(), "an lse that sees a NaN is not NaN"
    assert torch.equal(o[~hit], co[~hit]) and torch.equal(lse[~hit], cl[~hit])


def _some_rows(n, hq):
    hit = torch.zeros(n, hq, dtype=torch.bool)
    hit[0, 1] = hit[n // 2, hq - 1] = hit[n - 1, 0] = True
    return hit


def _sinks(hq, on):
    return torch.linspace(-2, 2, hq, device=DEV) if on else None


# ------------------------------------------------------ extend, 4-bit pool
@pytest.mark.parametrize("prefix,extend", LENGTHS)
@pytest.mark.parametrize("d,window,first,sinks", [(128, -1, 0, False), (64, 700, 4, True)])
def test_extend_fp4_nan_query(prefix, extend, d, window, first, sinks):
    c = Case(d, 8, 2, prefix, extend, 21, 0.3, 0.7)
    run = lambda: c.run(0.0, window, first, _sinks(8, sinks))[:2]
    clean = run()
    hit = _some_rows(c.q.shape[0], 8)
    c.q[..., 5][hit.to(DEV)] = NAN
    _check(run(), clean, hit)


@pytest.mark.parametrize("prefix,extend,seq,key", [
    ([100, 0, 300], [20, 5, 3], 0, 40), ([150] * 160, [2] * 160, 7, 149), ([8000], [3], 0, 5000),
    ([6000, 10, 0], [70, 300, 2], 0, 5990), ([6000, 10, 0], [70, 300, 2], 1, 3)])
@pytest.mark.parametrize("window,first,sinks", [(-1, 0, False), (40, 2, True)])
def test_extend_fp4_nan_block(prefix, extend, seq, key, window, first, sinks):
    """A block of a K row whose scale is NaN, seen by the group's heads, and
    with a window by those rows alone that still see the key."""
    c = Case(128, 8, 2, prefix, extend, 22, 0.3, 0.7)
    run = lambda: c.run(0.0, window, first, _sinks(8, sinks))[:2]
    clean = run()
    c.pool[1].view(torch.uint8)[int(c.wl.kv_indices[sum(prefix[:seq]) + key]), 1, 3] = 0x7F
    hit = torch.zeros(c.q.shape[0], 8, dtype=torch.bool)
    pos = prefix[seq] + torch.arange(extend[seq])
    sees = (pos - key <= window) | (key < first) if window > 0 else torch.ones_like(pos, dtype=torch.bool)
    hit[sum(extend[:seq]):sum(extend[:seq + 1]), 4:] = sees[:, None]
    _check(run(), clean, hit)


# ------------------------------------------------------- streaming, bf16 pool
@pytest.mark.parametrize("prefix,extend", LENGTHS)
@pytest.mark.parametrize("d,sinks", [(128, False), (64, True)])
def test_streaming_extend_nan_query(prefix, extend, d, sinks):
    c = Extend(W.draw(W.small_spec(batch=len(prefix), hq=8, hkv=2, lq=d, lv=d, prefix=prefix, extend=extend,
                                   seed=23)))
    run = lambda: c.run(900, 4, 0.0, _sinks(8, sinks))[:2]
    clean = run()
    hit = _some_rows(c.q.shape[0], 8)
    c.q[..., 5][hit.to(DEV)] = NAN
    _check(run(), clean, hit)


def _streaming_decode(wl, q, k, v, window, first):
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    pkx.decode_attention_fwd_streaming(q, o, k, v, wl.kv_indptr.to(DEV), wl.kv_indices.to(DEV), window, first,
                                       wl.sm_scale, lse=lse)
    return o, lse


@pytest.mark.parametrize("lens", DECODE_LENGTHS)
@pytest.mark.parametrize("d,hq,hkv,window,first", [(128, 8, 2, 600, 4), (64, 16, 1, 5000, 70)])
def test_streaming_decode_nan(lens, d, hq, hkv, window, first):
    """A NaN query, then a NaN key of the first tokens or of the window: one
    tile (the second key stream has none), several, split ones."""
    wl = W.draw(W.small_spec(batch=len(lens), hq=hq, hkv=hkv, lq=d, lv=d, prefix=lens, extend=[0] * len(lens),
                             seed=24, decode=True))
    q, (k, v) = wl.q.to(DEV), wl.pool(DEV)
    clean = _streaming_decode(wl, q, k, v, window, first)
    some = [b for b, t in enumerate(lens) if t]  # (a sequence without keys reads no query)
    hit = torch.zeros(len(lens), hq, dtype=torch.bool)
    hit[some[0], 1] = hit[some[-1], hq - 1] = True
    bad = q.clone()
    bad[..., 5][hit.to(DEV)] = NAN
    _check(_streaming_decode(wl, bad, k, v, window, first), clean, hit)
    for key in (0, lens[some[-1]] - 1):
        b = some[-1]
        kk = k.clone()
        kk[int(wl.kv_indices[int(wl.kv_indptr[b]) + key]), hkv - 1, d - 1] = NAN
        hit = torch.zeros(len(lens), hq, dtype=torch.bool)
        hit[b, hq - hq // hkv:] = True
        _check(_streaming_decode(wl, q, kk, v, window, first), clean, hit)


# -------------------------------------------- the forms they share the code with
MLA = dict(hq=16, hkv=1, lq=576, lv=512, v_aliases_k=True)


@pytest.mark.parametrize("form", ["extend", "unified", "ragged_paged"])
@pytest.mark.parametrize("heads", [dict(hq=8, hkv=2, lq=128, lv=128), dict(hq=8, hkv=8, lq=64, lv=64), MLA,
                                   dict(hq=8, hkv=4, lq=192, lv=128)], ids=lambda h: f"{h['lq']}")
@pytest.mark.parametrize("prefix,extend", [LENGTHS[i] for i in (0, 1, 3)])
def test_extend_forms_nan_query(form, heads, prefix, extend):
    w = DeviceWorkload(W.draw(W.small_spec(batch=len(prefix), prefix=prefix, extend=extend, seed=25, **heads)))
    run = lambda: getattr(w, form)()[:2]
    clean = run()
    hit = _some_rows(w.q.shape[0], heads["hq"])
    w.q[..., 5][hit.to(DEV)] = NAN
    _check(run(), clean, hit)


@pytest.mark.parametrize("heads", [dict(hq=8, hkv=2, lq=128, lv=128), dict(hq=8, hkv=8, lq=64, lv=64), MLA,
                                   dict(hq=8, hkv=4, lq=192, lv=128)], ids=lambda h: f"{h['lq']}")
@pytest.mark.parametrize("lens", DECODE_LENGTHS)
def test_decode_nan_query(heads, lens):
    w = DeviceWorkload(W.draw(W.small_spec(batch=len(lens), prefix=lens, extend=[0] * len(lens), seed=26, decode=True,
                                           **heads)))
    clean = w.decode()[:2]
    some = [b for b, t in enumerate(lens) if t]
    hit = torch.zeros(len(lens), heads["hq"], dtype=torch.bool)
    hit[some[0], 1] = hit[some[-1], heads["hq"] - 1] = True
    w.q[..., 5][hit.to(DEV)] = NAN
    _check(w.decode()[:2], clean, hit)


@pytest.mark.parametrize("lens", DECODE_LENGTHS)
def test_decode_fp8_nan_query(lens):
    wl = W.draw(W.small_spec(batch=len(lens), prefix=lens, extend=[0] * len(lens), seed=27, decode=True))
    k, v = wl.pool_fp8(torch.float8_e4m3fn, 0.05, 0.04, DEV)
    q, ptr, idx = (x.to(DEV) for x in (wl.q, wl.kv_indptr, wl.kv_indices))

    def run(q):
        o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=DEV)
        pkx.decode_attention_fwd(q, o, k, v, ptr, idx, wl.sm_scale, lse=lse, k_scale=0.05, v_scale=0.04)
        return o, lse

    clean = run(q)
    some = [b for b, t in enumerate(lens) if t]
    hit = torch.zeros(q.shape[:2], dtype=torch.bool)
    hit[some[0], 1] = hit[some[-1], 7] = True
    bad = q.clone()
    bad[..., 5][hit.to(DEV)] = NAN
    _check(run(bad), clean, hit)
