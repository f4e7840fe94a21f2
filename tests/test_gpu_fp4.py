"""GPU tests of the 4-bit KV pool: the quantising write bit-exact, the read
back bit-exact, decode attention over the pool, against the plain float64
implementation in fp4_reference.py."""
import math

import pytest
import torch

import fp4_reference as R
from paged_kv_extend_gb300 import pkx

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F16_STEP = 2.0 ** -11  # half a step of f16, which P is rounded to


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkx.load_library()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _bf16(g, *shape, amp=1.0):
    return (torch.randn(*shape, generator=g) * amp).bfloat16()


def _random_pool(g, slots, hkv, d):
    """Codes of every kind and block scales of a normal cache's size, on the CPU."""
    codes = torch.randint(0, 256, (slots, hkv, d // 2), generator=g, dtype=torch.uint8)
    bscale = torch.randint(0x20, 0x34, (slots, hkv, d // 16), generator=g, dtype=torch.uint8)
    return codes, bscale


def _to_dev(codes, bscale):
    return codes.to(DEV), bscale.view(torch.float8_e4m3fn).to(DEV)


# ------------------------------------------------------------------- write
@pytest.mark.parametrize("n,hkv,lk,lv,ks,vs,amp", [
    (1, 1, 64, 64, 1.0, 1.0, 1.0), (77, 8, 128, 128, 0.373, 2.5, 3.0), (130, 3, 64, 64, 1.0, 1.0, 1e-3),
    (63, 2, 16, 48, 1.0, 0.7, 2e4), (19, 1, 576, 512, 0.051, 1.0, 1.0), (700, 5, 128, 64, 3.1, 1.0, 40.0),
    (5000, 3, 64, 128, 0.125, 2.0 ** 20, 5.0), (33, 40, 128, 128, 2.0 ** -64, 2.0 ** 64, 1.0),
    (33, 2, 128, 128, 2.0 ** -65, 2.0 ** 65, 1e-19), (9, 64, 256, 48, 1.0, 1.0, 1.0),
])
def test_write_bit_exact(n, hkv, lk, lv, ks, vs, amp):
    """Codes and block scales of every row; strided inputs; slots that are
    not written keep their bytes; a slot outside the pool is skipped."""
    g = _gen(n + lk)
    slots = 2 * n + 5
    k = _bf16(g, n, hkv + 1, lk, amp=amp)[:, 1:]
    v = _bf16(g, n, hkv, lv, amp=amp)
    loc = torch.randperm(slots, generator=g)[:n]
    if n > 2:
        loc[n // 2] = slots + 3
        loc[n - 1] = -1
    kc, kb = _random_pool(g, slots, hkv, lk)
    vc, vb = _random_pool(g, slots, hkv, lv)
    want = [x.clone() for x in (kc, kb, vc, vb)]
    ok = (loc >= 0) & (loc < slots)
    for i, (x, s) in enumerate(((k, ks), (v, vs))):
        c, b = R.pack(x, s)
        want[2 * i][loc[ok]], want[2 * i + 1][loc[ok]] = c[ok], b[ok]
    pool = *_to_dev(kc, kb), *_to_dev(vc, vb)
    dk = torch.zeros(n, hkv + 1, lk, dtype=torch.bfloat16, device=DEV)[:, 1:]
    dk.copy_(k)
    pkx.set_kv_buffer_fp4(*pool, loc.to(DEV), dk, v.to(DEV), ks, vs)
    for got, w in zip(pool, want):
        assert torch.equal(got.view(torch.uint8).cpu(), w)


def test_write_borders():
    """Every midpoint and its neighbours, zeros of both signs, values below
    the smallest scale, infinities and NaN."""
    rows = []
    for s in (1.0, 1.125, 448.0, 2.0 ** -9, 2.0 ** -6 * 1.5):
        mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
        vals = [6.0 * s] + [m * s for m in mids] + [-m * s for m in mids] + [0.0]
        rows.append(vals)
        rows.append([6.0 * s] + [m * s * (1 + 2.0 ** -7) for m in mids] +
                    [-m * s * (1 - 2.0 ** -8) for m in mids] + [-0.0])
    inf, nan = float("inf"), float("nan")
    rows += [[0.0] * 16, [-0.0] * 16, [1e-30] * 15 + [-1e-30], [2.0 ** -8] * 16,
             [inf] + [1.0] * 14 + [-inf], [nan] + [1.0] * 15, [1.0] * 8 + [nan, inf] + [-2.0] * 6,
             [3e38] * 8 + [-3e38] * 8, [6.375 * 2.0 ** i for i in range(-8, 8)]]
    x = torch.tensor(rows).bfloat16()[:, None]  # [n, 1, 16]
    n = x.shape[0]
    for scale in (1.0, 0.37, 2.0 ** -7, 64.0):
        c, b = R.pack(x, scale)
        kc = torch.zeros(n, 1, 8, dtype=torch.uint8, device=DEV)
        kb = torch.zeros(n, 1, 1, dtype=torch.float8_e4m3fn, device=DEV)
        pkx.set_kv_buffer_fp4(kc, kb, None, None, torch.arange(n, device=DEV), x.to(DEV),
                              k_scale=scale)
        assert torch.equal(kb.view(torch.uint8).cpu(), b)
        assert torch.equal(kc.cpu(), c)
    assert int(b[-4]) == 0x7F and int(b[-3]) == 0x7F  # the rows with a NaN


@pytest.mark.parametrize("scale", [1.0, 4.0, 0.3])
def test_write_every_bf16(scale):
    """Every finite bf16 next to block maxima of all mantissas, so that every
    quotient of a value and a block scale is met at all its roundings."""
    g = _gen(17)
    bits = torch.arange(0x0080, 0x7F80, dtype=torch.int32)
    vals = bits.to(torch.int16).view(torch.bfloat16)
    near = vals[(vals > 2.0 ** -12) & (vals < 2.0 ** 12)]
    n = 60000
    top = near[torch.randint(0, near.numel(), (n,), generator=g)].float()
    x = (top[:, None] * torch.rand(n, 16, generator=g)).bfloat16()
    x[:, 0] = top.bfloat16()
    x[:, 1] = vals[torch.randint(0, vals.numel(), (n,), generator=g)]
    x = (x.float() * (torch.randint(0, 2, x.shape, generator=g) * 2 - 1)).bfloat16()[:, None]
    c, b = R.pack(x, scale)
    kc = torch.zeros(n, 1, 8, dtype=torch.uint8, device=DEV)
    kb = torch.zeros(n, 1, 1, dtype=torch.float8_e4m3fn, device=DEV)
    pkx.set_kv_buffer_fp4(kc, kb, None, None, torch.arange(n, device=DEV), x.to(DEV), k_scale=scale)
    assert torch.equal(kb.view(torch.uint8).cpu(), b) and torch.equal(kc.cpu(), c)


def test_write_nothing():
    kc = torch.zeros(4, 2, 32, dtype=torch.uint8, device=DEV)
    kb = torch.zeros(4, 2, 4, dtype=torch.float8_e4m3fn, device=DEV)
    empty = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    pkx.set_kv_buffer_fp4(kc, kb, kc.clone(), kb.clone(), torch.zeros(0, dtype=torch.int64, device=DEV),
                          empty, empty)
    assert not kc.any()


# --------------------------------------------------------------- read back
@pytest.mark.parametrize("n,hkv,lk,lv,ks,vs", [
    (1, 1, 64, 64, 1.0, 1.0), (333, 3, 64, 128, 0.373, 2.5), (40, 8, 128, 128, 1.0, 1.0),
    (51, 1, 576, 512, 0.051, 7.0), (7, 2, 16, 48, 1.0, 1.0)])
def test_read_bit_exact(n, hkv, lk, lv, ks, vs):
    """bf16 of the fp32 product, bit for bit; a slot outside the pool reads
    zero; strided outputs; repeated slots; block scales of every code."""
    g = _gen(n)
    slots = n + 9
    kc, kb = _random_pool(g, slots, hkv, lk)
    vc, vb = _random_pool(g, slots, hkv, lv)
    vb = torch.randint(0, 127, vb.shape, generator=g, dtype=torch.uint8)  # no NaN
    idx = torch.randint(0, slots, (n,), generator=g, dtype=torch.int32)
    if n > 4:
        idx[3], idx[4] = -7, slots
    bad = (idx < 0) | (idx >= slots)
    out = torch.zeros(n, 2 * hkv, lk + 8, dtype=torch.bfloat16, device=DEV)
    k_out = out[:, ::2, :lk]
    k, v = pkx.get_kv_buffer_fp4(*_to_dev(kc, kb), *_to_dev(vc, vb), idx.to(DEV), ks, vs, k_out=k_out)
    assert k is k_out and not out[:, 1::2].any() and not out[:, :, lk:].any()
    for got, c, b, s in ((k, kc, kb, ks), (v, vc, vb, vs)):
        w = R.unpack(c, b).float()[idx.long().clamp(0, slots - 1)] * torch.tensor(s, dtype=torch.float32)
        w[bad] = 0.0
        assert torch.equal(got.cpu(), w.bfloat16())
    k2, v2 = pkx.get_kv_buffer_fp4(*_to_dev(kc, kb), None, None, idx.to(DEV), ks)
    assert v2 is None and torch.equal(k2, k)


def test_read_nan_block():
    kc = torch.full((1, 1, 16), 0x21, dtype=torch.uint8)
    kb = torch.tensor([[[0x7F, 0x38]]], dtype=torch.uint8)
    k, _ = pkx.get_kv_buffer_fp4(*_to_dev(kc, kb), None, None, torch.zeros(1, dtype=torch.int32, device=DEV))
    assert torch.isnan(k[..., :16]).all() and torch.equal(k[0, 0, 16:18].cpu().float(), torch.tensor([0.5, 1.0]))


# ------------------------------------------------------------------ decode
class Decode:
    def __init__(self, d, hq, hkv, lens, seed, ks=1.0, vs=1.0, qamp=1.0):
        g = _gen(seed)
        self.d, self.hq, self.hkv, self.lens, self.ks, self.vs = d, hq, hkv, lens, ks, vs
        total = sum(lens)
        slots = total + total // 3 + 8
        self.k, self.v = _random_pool(g, slots, hkv, d), _random_pool(g, slots, hkv, d)
        self.idx = torch.randperm(slots, generator=g)[:total].to(torch.int32)
        self.q = _bf16(g, len(lens), hq, d, amp=qamp)
        self.indptr = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)
        self.scale = d ** -0.5
        self.dev = [x.to(DEV) for x in (*_to_dev(*self.k), *_to_dev(*self.v), self.indptr, self.idx)]

    def run(self, cap=0.0, window=-1, first=0, ws=None, q=None, **over):
        q = self.q.to(DEV) if q is None else q
        o = torch.full_like(q, float("nan"))
        lse = torch.full(q.shape[:2], float("nan"), device=DEV)
        kc, kb, vc, vb, ptr, idx = self.dev
        a = dict(kc=kc, kb=kb, vc=vc, vb=vb, idx=idx)
        a.update(over)
        ws = pkx.decode_attention_fwd_fp4(q, o, a["kc"], a["kb"], a["vc"], a["vb"], ptr, a["idx"], self.scale,
                                          cap, window, first, lse, ws, self.ks, self.vs)
        return o, lse, ws

    def reference(self, cap=0.0, window=-1, first=0):
        out, k0 = [], 0
        for b, t in enumerate(self.lens):
            at = self.idx[k0:k0 + t].long()
            k = R.unpack(self.k[0][at], self.k[1][at], self.ks)
            v = R.unpack(self.v[0][at], self.v[1][at], self.vs)
            ok = R.visible(torch.tensor([t - 1]), t, window, first)
            out.append(R.attend(self.q[b:b + 1].double(), k, v, ok, self.scale, cap))
            k0 += t
        return [torch.cat(x) for x in zip(*out)]


@pytest.mark.parametrize("d,hq,hkv,lens,cap,window,first,ks,vs", [
    (128, 32, 8, [1, 0, 31, 32, 33, 64, 500], 0.0, -1, 0, 1.0, 1.0),
    (64, 12, 3, [777, 1, 0, 129], 0.0, -1, 0, 0.37, 2.5),
    (128, 28, 4, [900, 45, 3000, 2], 20.0, 100, 4, 0.05, 0.02),
    (64, 16, 1, [5000, 17], 0.0, 64, 1, 0.5, 1.0),          # two column tiles of heads, 16 shares a CTA
    (128, 64, 4, [700, 0, 65], 0.0, 33, 40, 1.0, 1.0),      # group 16
    (128, 40, 2, [300, 129], 5.0, -1, 0, 0.25, 0.5),        # group 20: the last column tile is part full
    (64, 128, 1, [260, 31], 0.0, 31, 0, 1.0, 1.0),          # group 128
    (128, 24, 24, [70, 300, 0, 0, 5], 0.0, -1, 0, 1.0, 1.0),  # group 1, more heads than warps
    (64, 5, 5, [40] * 9 + [1] * 5, 0.0, 7, 3, 1.0, 3.0),
    (128, 8, 1, [20000], 0.0, -1, 0, 1.0, 1.0),             # one sequence over the whole device
    (128, 32, 8, [16384, 3, 0, 40000], 0.0, -1, 0, 0.1, 0.3),
    (64, 8, 2, [1] * 700, 0.0, -1, 0, 1.0, 1.0),            # more sequences than threads
    (128, 4, 1, [50, 60], 0.0, 1000, 10, 1.0, 1.0),         # a window longer than the keys
    (128, 8, 2, [400, 33], 0.0, 100, 100000, 1.0, 1.0),     # first tokens past the keys
    (128, 8, 2, [700, 33], 0.0, -1, 0, 2.0 ** -64, 2.0 ** 64),   # the scales' limits
    (64, 8, 2, [700, 33], 3.0, -1, 0, 2.0 ** -64, 2.0 ** -64),
])
def test_decode(d, hq, hkv, lens, cap, window, first, ks, vs):
    c = Decode(d, hq, hkv, lens, seed=d + hq + sum(lens), ks=ks, vs=vs)
    o, lse, ws = c.run(cap, window, first)
    R.check(o, lse, c.reference(cap, window, first), d, c.scale * 1.0, F16_STEP, f"{lens}")
    assert pkx.workspace_status(ws) == 0


@pytest.mark.parametrize("d,hq,hkv,lens,at,nats", [
    (128, 8, 2, [3000, 40], 0, 17.0), (64, 12, 4, [900, 2000], 500, 17.0), (128, 16, 1, [30000], 3, 14.0)])
def test_decode_dominant_key_with_a_zero_value(d, hq, hkv, lens, at, nats):
    """One key takes nearly all of the weight and its value is zero, so that
    the output is made of keys with weights of 2^-20 to 2^-25: they keep P's
    11 bits."""
    c = Decode(d, hq, hkv, lens, seed=d + at)
    g = _gen(at)
    slots = c.k[0].shape[0]
    c.q = _bf16(g, 1, hkv, 1, d).expand(len(lens), hkv, hq // hkv, d).reshape(len(lens), hq, d).contiguous()
    k, v = _bf16(g, slots, hkv, d, amp=0.1), _bf16(g, slots, hkv, d) + 0.5
    q = c.q[0].float().view(hkv, hq // hkv, d)[:, 0]
    for b in range(len(lens)):
        slot = int(c.idx[int(c.indptr[b]) + min(at, lens[b] - 1)])
        k[slot] = (q * (nats / c.scale / q.square().sum(-1, keepdim=True))).bfloat16()
        v[slot] = 0
    c.k, c.v = R.pack(k, 1.0), R.pack(v, 1.0)
    c.dev[:4] = [x.to(DEV) for x in (*_to_dev(*c.k), *_to_dev(*c.v))]
    o, lse, _ = c.run()
    R.check(o, lse, c.reference(), d, c.scale, F16_STEP)


@pytest.mark.parametrize("qamp", [1e-20, 3e-3, 60.0])
def test_decode_query_range(qamp):
    """Queries far outside f16's range keep their bits."""
    c = Decode(128, 8, 2, [70, 9, 200], seed=5, qamp=qamp)
    c.scale = 0.05 / qamp
    o, lse, _ = c.run()
    R.check(o, lse, c.reference(), 128, c.scale, F16_STEP)


def test_decode_query_of_the_largest_exponent():
    c = Decode(128, 8, 2, [70, 9], seed=12)
    c.q[0, 3, 5], c.q[1, 7, 64], c.q[1, 7, 66] = 3.2e38, -2.5e38, 1e36
    c.scale = 2e-38
    o, lse, _ = c.run()
    R.check(o, lse, c.reference(), 128, c.scale, F16_STEP)


def test_decode_zero_query_and_zero_pool():
    """All logits 0: the mean of the values; a pool of zeros gives zeros."""
    c = Decode(128, 8, 2, [100, 33], seed=6)
    o, lse, _ = c.run(q=torch.zeros(2, 8, 128, dtype=torch.bfloat16, device=DEV))
    assert torch.allclose(lse.cpu(), torch.tensor([100.0, 33.0]).log()[:, None].expand(2, 8), atol=1e-5)
    zero = torch.zeros_like(c.dev[2])
    o, _, _ = c.run(vc=zero)
    assert not o.any()


def test_decode_nan_and_inf_stay_in_their_row():
    """A NaN block of a visible key reaches its sequence's heads only; one
    outside the window and the first tokens reaches nothing."""
    c = Decode(128, 8, 2, [200, 90, 33], seed=7)
    clean, _, _ = c.run()
    kb = c.dev[1].view(torch.uint8).clone()
    kb[int(c.idx[200 + 5]), 1, 3] = 0x7F  # key 5 of sequence 1, KV head 1
    o, lse, _ = c.run(kb=kb.view(torch.float8_e4m3fn))
    assert torch.isnan(o[1, 4:]).all() and torch.isnan(lse[1, 4:]).all()
    assert torch.equal(o[1, :4], clean[1, :4]) and torch.equal(o[[0, 2]], clean[[0, 2]])
    o, lse, _ = c.run(kb=kb.view(torch.float8_e4m3fn), window=20, first=5)
    want, wl, _ = c.run(window=20, first=5)
    assert torch.equal(o, want) and torch.equal(lse, wl)


def test_decode_bad_slot_reads_zero_and_is_reported():
    c = Decode(64, 8, 2, [40, 70], seed=8)
    idx = c.dev[5].clone()
    idx[45], idx[50] = 1 << 30, -3
    o, lse, ws = c.run(idx=idx)
    assert pkx.workspace_status(ws) == pkx.PKX_EDEVICE
    at = c.idx.clone()
    k, v = R.unpack(c.k[0][at.long()], c.k[1][at.long()]), R.unpack(c.v[0][at.long()], c.v[1][at.long()])
    for i in (45, 50):
        k[i] = 0.0
        v[i] = 0.0
    ref = R.attend(c.q[1:].double(), k[40:], v[40:], torch.ones(1, 70, dtype=torch.bool), c.scale)
    R.check(o[1:], lse[1:], ref, 64, c.scale, F16_STEP)
    _, _, ws = c.run(ws=ws)  # the next call's status is its own
    assert pkx.workspace_status(ws) == 0


def test_decode_strided_interleaved_pool():
    """Codes and block scales of K and V in one tensor, one row after another."""
    c = Decode(128, 16, 4, [333, 20], seed=9)
    slots = c.k[0].shape[0]
    big = torch.zeros(slots, 4, 160, dtype=torch.uint8, device=DEV)
    kc, vc = big[:, :, :64], big[:, :, 80:144]
    kb, vb = (big[:, :, a:a + 8].view(torch.float8_e4m3fn) for a in (64, 144))
    kc.copy_(c.dev[0]), vc.copy_(c.dev[2])
    big[:, :, 64:72].copy_(c.dev[1].view(torch.uint8)), big[:, :, 144:152].copy_(c.dev[3].view(torch.uint8))
    want, wl, _ = c.run()
    o, lse, _ = c.run(kc=kc, kb=kb, vc=vc, vb=vb)
    assert torch.equal(o, want) and torch.equal(lse, wl)


def test_decode_repeats_and_streams_and_graph():
    """The same call twice, on another stream, and captured and replayed with
    new inputs, bit for bit; a graph's calls share one workspace."""
    c = Decode(128, 32, 8, [3000, 1, 250, 700], seed=10)
    want, wl, ws = c.run(window=900, first=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, lse, _ = c.run(window=900, first=4)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, want) and torch.equal(lse, wl)
    q = torch.zeros_like(want)
    kc, kb, vc, vb, ptr, idx = c.dev
    outs = [torch.zeros_like(want) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for o, w in zip(outs, (900, -1)):
            pkx.decode_attention_fwd_fp4(q, o, kc, kb, vc, vb, ptr, idx, c.scale, 0.0, w, 4, None, ws)
    q.copy_(c.q)
    graph.replay()
    graph.replay()
    full, _, _ = c.run()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], full)


@pytest.mark.parametrize("hq,hkv,long", [(32, 4, []), (8, 1, [30000, 7, 25000])])
def test_decode_many_split_sequences(hq, hkv, long):
    """More sequences that several shares hold than a CTA of the merge takes
    rows: every one is merged, in repeated calls on one workspace.  One KV
    head: 16 shares a CTA, and some sequences of more than 32 parts."""
    c = Decode(64, hq, hkv, [700 + 13 * i for i in range(90)] + long, seed=15)
    ref, ws = c.reference(), None
    for _ in range(20):
        o, lse, ws = c.run(ws=ws)
        R.check(o, lse, ref, 64, c.scale, F16_STEP)


def test_write_then_decode():
    """A decode step as a serving loop runs it: the new token is written, then
    read by the attention, over several steps."""
    g = _gen(11)
    d, hq, hkv, b, slots = 128, 16, 4, 3, 400
    pool = (torch.zeros(slots, hkv, d // 2, dtype=torch.uint8, device=DEV),
            torch.zeros(slots, hkv, d // 16, dtype=torch.float8_e4m3fn, device=DEV))
    pool = (*pool, pool[0].clone(), pool[1].clone())
    free = torch.randperm(slots, generator=g)
    owned, rows, ws = [[] for _ in range(b)], [[] for _ in range(b)], None
    ks, vs = 0.21, 0.4
    for step in range(40):
        k, v, q = _bf16(g, b, hkv, d), _bf16(g, b, hkv, d), _bf16(g, b, hq, d)
        loc = free[step * b:(step + 1) * b]
        pkx.set_kv_buffer_fp4(*pool, loc.to(DEV), k.to(DEV), v.to(DEV), ks, vs)
        for i in range(b):
            owned[i].append(int(loc[i]))
            rows[i].append((k[i], v[i]))
        ptr = torch.arange(b + 1, dtype=torch.int32) * (step + 1)
        idx = torch.tensor([s for o in owned for s in o], dtype=torch.int32)
        o = torch.empty(b, hq, d, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(b, hq, device=DEV)
        ws = pkx.decode_attention_fwd_fp4(q.to(DEV), o, *pool, ptr.to(DEV), idx.to(DEV), None, 0.0, 16, 2,
                                          lse, ws, ks, vs)
        if step % 13 == 0:
            for i in range(b):
                kk = R.unpack(*R.pack(torch.stack([r[0] for r in rows[i]]), ks), ks)
                vv = R.unpack(*R.pack(torch.stack([r[1] for r in rows[i]]), vs), vs)
                ok = R.visible(torch.tensor([step]), step + 1, 16, 2)
                ref = R.attend(q[i:i + 1].double(), kk, vv, ok, 1 / math.sqrt(d))
                R.check(o[i:i + 1], lse[i:i + 1], ref, d, 1 / math.sqrt(d), F16_STEP)


def test_offsets_past_32_bits():
    """Slots whose bytes lie past 4 GB in every tensor of the pool: write, read
    back, decode and extend."""
    g = _gen(16)
    d, hq, hkv, n, step = 128, 8, 2, 40, 1 << 27  # slots 128 MB apart
    big = torch.zeros(n * step + 4096, dtype=torch.uint8, device=DEV)
    at = lambda off, w: big[off:].as_strided((n, hkv, w), (step, w, 1))
    kc, vc = at(0, d // 2), at(512, d // 2)
    kb, vb = (at(o, d // 16).view(torch.float8_e4m3fn) for o in (1024, 1536))
    k, v = _bf16(g, n, hkv, d), _bf16(g, n, hkv, d)
    loc = torch.randperm(n, generator=g)
    pkx.set_kv_buffer_fp4(kc, kb, vc, vb, loc.to(DEV), k.to(DEV), v.to(DEV))
    kk, vv = R.unpack(*R.pack(k, 1.0)), R.unpack(*R.pack(v, 1.0))
    idx = loc.to(torch.int32).to(DEV)
    gk, gv = pkx.get_kv_buffer_fp4(kc, kb, vc, vb, idx)
    assert torch.equal(gk.cpu(), kk.bfloat16()) and torch.equal(gv.cpu(), vv.bfloat16())
    q, e = _bf16(g, 1, hq, d), _bf16(g, 3, hq, d)
    ke, ve = _bf16(g, 3, hkv, d), _bf16(g, 3, hkv, d)
    ptr = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    o, lse = torch.empty(1, hq, d, dtype=torch.bfloat16, device=DEV), torch.empty(1, hq, device=DEV)
    pkx.decode_attention_fwd_fp4(q.to(DEV), o, kc, kb, vc, vb, ptr, idx, lse=lse)
    ok = torch.ones(1, n, dtype=torch.bool)
    R.check(o, lse, R.attend(q.double(), kk, vv, ok, d ** -0.5), d, d ** -0.5, F16_STEP)
    o, lse = torch.empty(3, hq, d, dtype=torch.bfloat16, device=DEV), torch.empty(3, hq, device=DEV)
    qo = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    pkx.extend_attention_fwd_fp4(e.to(DEV), ke.to(DEV), ve.to(DEV), o, kc, kb, vc, vb, qo, ptr, idx, lse=lse)
    ref = R.attend(e.double(), torch.cat([kk, ke.double()]), torch.cat([vv, ve.double()]),
                   R.visible(torch.arange(3) + n, n + 3, -1, 0), d ** -0.5)
    R.check(o, lse, ref, d, d ** -0.5, 2.0 ** -8)


def test_decode_wait_that_runs_out_is_reported():
    """The stall hook makes a wait run out: the status says so, the context
    stays usable and the next call is whole again."""
    c = Decode(128, 32, 8, [4000, 900], seed=18)
    want, wl, _ = c.run()
    pkx.set_wait_limit_ns(20_000_000)
    pkx.set_stall_injection(True)
    try:
        _, _, ws = c.run()
        assert pkx.workspace_status(ws) == pkx.PKX_ETIMEOUT
    finally:
        pkx.set_stall_injection(False)
        pkx.set_wait_limit_ns(0)
    o, lse, ws = c.run(ws=ws)
    assert pkx.workspace_status(ws) == 0 and torch.equal(o, want) and torch.equal(lse, wl)
