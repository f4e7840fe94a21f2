"""GPU tests of extend attention over a 4-bit pool against the plain float64
implementation in fp4_reference.py: the prefix as the pool holds it, the new
rows in bf16."""
import pytest
import torch

import fp4_reference as R
from paged_kv_extend_gb300 import pkx
from paged_kv_extend_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16_STEP = 2.0 ** -8   # half a step of bf16, which P is rounded to
TANH_STEP = 2.0 ** -11  # tanh.approx


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkx.load_library()


class Case:
    def __init__(self, d, hq, hkv, prefix, extend, seed, ks=1.0, vs=1.0):
        self.wl = wl = W.draw(W.small_spec(batch=len(prefix), hq=hq, hkv=hkv, lq=d, lv=d, prefix=prefix,
                                           extend=extend, seed=seed))
        self.ks, self.vs = ks, vs
        at = torch.cat([torch.arange(int(wl.token_offsets[b]), int(wl.token_offsets[b]) + p)
                        for b, p in enumerate(prefix)])
        slots = wl.spec.num_slots
        pool, self.rows = [], []
        for rows, s in ((wl.k_rows, ks), (wl.v_rows, vs)):
            c, b = R.pack(rows[at], s) if len(at) else (torch.zeros(0, hkv, d // 2, dtype=torch.uint8),
                                                        torch.zeros(0, hkv, d // 16, dtype=torch.uint8))
            self.rows.append(R.unpack(c, b, s))
            codes = torch.full((slots, hkv, d // 2), 0x7F, dtype=torch.uint8)
            scales = torch.full((slots, hkv, d // 16), 0x7F, dtype=torch.uint8)  # NaN in every other slot
            codes[wl.kv_indices.long()], scales[wl.kv_indices.long()] = c, b
            pool += [codes.to(DEV), scales.view(torch.float8_e4m3fn).to(DEV)]
        self.pool = pool
        self.ke, self.ve = wl.extend_kv(DEV)
        self.q, self.qo, self.ptr, self.idx = (x.to(DEV) for x in (wl.q, wl.qo_indptr, wl.kv_indptr, wl.kv_indices))

    def run(self, cap=0.0, window=-1, first=0, sinks=None, mask=None, mask_indptr=None, ws=None, pool=None,
            idx=None):
        o = torch.full_like(self.q, float("nan"))
        lse = torch.full(self.q.shape[:2], float("nan"), device=DEV)
        ws = pkx.extend_attention_fwd_fp4(
            self.q, self.ke, self.ve, o, *(pool or self.pool), self.qo, self.ptr,
            self.idx if idx is None else idx, self.wl.sm_scale, cap, window, first, lse, ws, mask, mask_indptr,
            sinks, self.ks, self.vs)
        return o, lse, ws

    def reference(self, cap=0.0, window=-1, first=0, sinks=None, masks=None):
        return R.extend(self.wl, *self.rows, self.ke.cpu(), self.ve.cpu(), window, first, cap, sinks, masks)


@pytest.mark.parametrize("d,hq,hkv,prefix,extend,cap,window,first,ks,vs,sinks", [
    (128, 32, 8, [0, 5, 300, 1000], [1, 40, 77, 130], 0.0, -1, 0, 1.0, 1.0, False),
    (128, 28, 4, [600, 0, 90, 3000], [200, 1, 19, 5], 20.0, 100, 0, 0.05, 0.02, True),
    (64, 12, 3, [0, 999, 45], [500, 2, 129], 0.0, 250, 0, 0.5, 2.0, False),
    (64, 8, 8, [40, 1300], [70, 33], 5.0, -1, 0, 0.25, 0.125, False),
    (128, 16, 4, [700, 60], [300, 900], 0.0, 128, 129, 0.3, 0.7, True),
    (64, 8, 2, [10, 2000], [1100, 64], 0.0, 7, 300, 1.0, 1.0, False),
    (128, 8, 1, [8000], [3], 0.0, 512, 64, 0.1, 0.1, False),
    (64, 64, 1, [3000, 17], [70, 1], 0.0, -1, 0, 0.07, 3.0, True),
    (128, 128, 1, [900, 128], [40, 1], 0.0, -1, 0, 1.0, 1.0, False),
    (128, 2, 2, [0], [129], 0.0, -1, 0, 1.0, 1.0, False),   # no prefix at all
    (128, 6, 2, [127, 128, 129], [1, 1, 1], 0.0, -1, 0, 2.0, 0.5, False),
    (128, 8, 2, [200, 0, 700], [30, 140, 1], 0.0, -1, 0, 2.0 ** -64, 2.0 ** 64, False),  # the scales' limits
    (64, 8, 2, [200, 0, 1000], [30, 140, 1], 0.0, 300, 0, 2.0 ** -64, 2.0 ** -64, True),
])
def test_extend(d, hq, hkv, prefix, extend, cap, window, first, ks, vs, sinks):
    c = Case(d, hq, hkv, prefix, extend, sum(prefix) + d, ks, vs)
    sk = torch.randn(hq, generator=torch.Generator().manual_seed(hq)) * 2 if sinks else None
    o, lse, ws = c.run(cap, window, first, sk.to(DEV) if sinks else None)
    R.check(o, lse, c.reference(cap, window, first, sk), d, c.wl.sm_scale, BF16_STEP,
            tanh_step=TANH_STEP if cap else 0.0)
    assert pkx.workspace_status(ws) == 0


@pytest.mark.parametrize("d,hq,hkv,prefix,extend,at,nats,sinks", [
    (128, 8, 2, [2000, 300], [40, 3], 0, 16.0, False), (64, 4, 4, [900, 5000], [1, 130], 200, 16.0, True)])
def test_dominant_key_with_a_zero_value(d, hq, hkv, prefix, extend, at, nats, sinks):
    """One key of the pool takes nearly all of the weight and its value is
    zero, so that the output is made of keys with weights near 2^-23: they
    keep P's bits."""
    c = Case(d, hq, hkv, prefix, extend, d)
    wl, g = c.wl, torch.Generator().manual_seed(d)
    q = torch.randn(hkv, 1, d, generator=g).bfloat16()
    wl.q[:] = q.expand(hkv, hq // hkv, d).reshape(hq, d)
    c.q = wl.q.to(DEV)
    k = (torch.randn(sum(prefix), hkv, d, generator=g) * 0.1).bfloat16()
    v = (torch.randn(sum(prefix), hkv, d, generator=g) + 0.5).bfloat16()
    q = q[:, 0].float()
    p0 = 0
    for p in prefix:
        k[p0 + at] = (q * (nats / wl.sm_scale / q.square().sum(-1, keepdim=True))).bfloat16()
        v[p0 + at] = 0
        p0 += p
    c.rows = []
    slots = wl.kv_indices.long().to(DEV)
    for i, x in enumerate((k, v)):
        codes, scales = R.pack(x, 1.0)
        c.rows.append(R.unpack(codes, scales, 1.0))
        c.pool[2 * i][slots] = codes.to(DEV)
        c.pool[2 * i + 1].view(torch.uint8)[slots] = scales.to(DEV)
    c.ke *= 0.05
    sk = torch.randn(hq, generator=g) if sinks else None
    o, lse, _ = c.run(sinks=sk.to(DEV) if sinks else None)
    R.check(o, lse, c.reference(sinks=sk), d, wl.sm_scale, BF16_STEP)


@pytest.mark.parametrize("d,window,sinks", [(128, -1, False), (64, 50, True)])
def test_extend_with_a_custom_mask(d, window, sinks):
    from gpu_cases import random_masks
    c = Case(d, 8, 2, [300, 0, 77], [17, 64, 130], 11, 0.4, 0.6)
    flat, ptr = random_masks(c.wl, 5)
    masks = [flat[int(ptr[b]):int(ptr[b + 1])].view(e, -1) for b, e in enumerate(c.wl.extend_lens)]
    sk = torch.randn(8, generator=torch.Generator().manual_seed(8)) if sinks else None
    o, lse, _ = c.run(0.0, window, 0, sk.to(DEV) if sinks else None, flat.to(DEV), ptr.to(DEV))
    R.check(o, lse, c.reference(0.0, window, 0, sk, masks), d, c.wl.sm_scale, BF16_STEP)
    with pytest.raises(pkx.PkxError) as e:
        c.run(0.0, 50, 4, None, flat.to(DEV), ptr.to(DEV))
    assert e.value.code == pkx.PKX_EUNSUPPORTED


def test_bad_slot_is_reported():
    c = Case(128, 8, 2, [200, 50], [20, 5], 12)
    idx = c.idx.clone()
    idx[210] = 1 << 29
    o, _, ws = c.run(idx=idx)
    assert pkx.workspace_status(ws) == pkx.PKX_EDEVICE
    want, _, ws = c.run(ws=ws)
    assert pkx.workspace_status(ws) == 0 and torch.equal(o[:20], want[:20])


def test_interleaved_pool_stream_and_graph():
    """Codes and block scales of K and V in one tensor; another stream; a
    captured call replayed with other queries."""
    c = Case(128, 16, 4, [333, 20, 0], [20, 150, 1], 13, 0.3, 0.4)
    want, wl_, ws = c.run()
    big = torch.zeros(c.pool[0].shape[0], 4, 160, dtype=torch.uint8, device=DEV)
    kc, vc = big[:, :, :64], big[:, :, 80:144]
    kb, vb = (big[:, :, a:a + 8].view(torch.float8_e4m3fn) for a in (64, 144))
    kc.copy_(c.pool[0]), vc.copy_(c.pool[2])
    big[:, :, 64:72].copy_(c.pool[1].view(torch.uint8)), big[:, :, 144:152].copy_(c.pool[3].view(torch.uint8))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, lse, _ = c.run(pool=(kc, kb, vc, vb))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, want) and torch.equal(lse, wl_)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkx.extend_attention_fwd_fp4(c.q, c.ke, c.ve, out, *c.pool, c.qo, c.ptr, c.idx, c.wl.sm_scale,
                                     workspace=ws, k_scale=c.ks, v_scale=c.vs)
    c.q.mul_(-1.0)
    graph.replay()
    neg, _, _ = c.run()
    assert torch.equal(out, neg)


def test_serving_turns():
    """Turns of a conversation as a server runs them: extend over the cached
    prefix, the new rows written to the pool, decode steps, the next turn; the
    last turn's prefix read back is what attention saw."""
    g = torch.Generator().manual_seed(14)
    d, hq, hkv, slots, ks, vs = 64, 8, 2, 600, 0.3, 0.2
    pool = (torch.zeros(slots, hkv, d // 2, dtype=torch.uint8, device=DEV),
            torch.zeros(slots, hkv, d // 16, dtype=torch.float8_e4m3fn, device=DEV))
    pool = (*pool, pool[0].clone(), pool[1].clone())
    free = torch.randperm(slots, generator=g).to(torch.int32)
    used, keys, vals = 0, torch.zeros(0, hkv, d), torch.zeros(0, hkv, d)
    scale = d ** -0.5
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    for turn in (40, 1, 130, 7):
        q, k, v = (torch.randn(turn, h, d, generator=g).bfloat16() for h in (hq, hkv, hkv))
        o, lse = torch.empty(turn, hq, d, dtype=torch.bfloat16, device=DEV), torch.empty(turn, hq, device=DEV)
        pkx.extend_attention_fwd_fp4(q.to(DEV), k.to(DEV), v.to(DEV), o, *pool, i32([0, turn]), i32([0, used]),
                                     free[:used].to(DEV), scale, 0.0, 64, 4, lse, k_scale=ks, v_scale=vs)
        kk, vv = (R.unpack(*R.pack(x.bfloat16(), s), s) if used else x.double()
                  for x, s in ((keys, ks), (vals, vs)))
        ref = R.attend(q.double(), torch.cat([kk, k.double()]), torch.cat([vv, v.double()]),
                       R.visible(torch.arange(turn) + used, used + turn, 64, 4), scale)
        R.check(o, lse, ref, d, scale, BF16_STEP, f"turn of {turn}")
        loc = free[used:used + turn].long().to(DEV)
        pkx.set_kv_buffer_fp4(*pool, loc, k.to(DEV), v.to(DEV), ks, vs)
        keys, vals, used = torch.cat([keys, k.float()]), torch.cat([vals, v.float()]), used + turn
        for _ in range(3):  # decode steps
            q, k, v = (torch.randn(1, h, d, generator=g).bfloat16() for h in (hq, hkv, hkv))
            pkx.set_kv_buffer_fp4(*pool, free[used:used + 1].long().to(DEV), k.to(DEV), v.to(DEV), ks, vs)
            keys, vals, used = torch.cat([keys, k.float()]), torch.cat([vals, v.float()]), used + 1
            o, lse = torch.empty(1, hq, d, dtype=torch.bfloat16, device=DEV), torch.empty(1, hq, device=DEV)
            pkx.decode_attention_fwd_fp4(q.to(DEV), o, *pool, i32([0, used]), free[:used].to(DEV), scale, 0.0, 64, 4,
                                         lse, None, ks, vs)
            kk, vv = (R.unpack(*R.pack(x.bfloat16(), s), s) for x, s in ((keys, ks), (vals, vs)))
            ref = R.attend(q.double(), kk, vv, R.visible(torch.tensor([used - 1]), used, 64, 4), scale)
            R.check(o, lse, ref, d, scale, 2.0 ** -11, "decode step")
    k, v = pkx.get_kv_buffer_fp4(*pool, free[:used].to(DEV), ks, vs)
    # bf16 of an fp32 product: within half a step of bf16 (and of fp32)
    for got, want in ((k, kk), (v, vv)):
        assert ((got.cpu().double() - want).abs() <= (2.0 ** -8 + 2.0 ** -23) * want.abs()).all()


def test_rows_behind_the_last_sequence_stay():
    """A padded batch: query rows past qo_indptr's end and sequences without
    new tokens."""
    c = Case(64, 8, 2, [100, 50], [20, 30], 19)
    want, wl_, _ = c.run()
    pad = lambda x: torch.cat([x, torch.ones(7, *x.shape[1:], dtype=x.dtype, device=DEV)])
    qo = torch.cat([c.qo, c.qo[-1:], c.qo[-1:]])
    ptr = torch.cat([c.ptr, c.ptr[-1:], c.ptr[-1:]])
    q = pad(c.q)
    o, lse = torch.full_like(q, 5.0), torch.full(q.shape[:2], 6.0, device=DEV)
    ws = pkx.extend_attention_fwd_fp4(q, pad(c.ke), pad(c.ve), o, *c.pool, qo, ptr, c.idx, c.wl.sm_scale, lse=lse)
    assert pkx.workspace_status(ws) == 0
    assert torch.equal(o[:50], want) and torch.equal(lse[:50], wl_)
    assert (o[50:] == 5.0).all() and (lse[50:] == 6.0).all()
