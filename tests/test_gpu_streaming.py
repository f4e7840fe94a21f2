"""GPU tests of the streaming window (a sliding window before which the first
tokens stay visible) over a bf16 pool, extend and decode, against the plain
float64 implementation in fp4_reference.py."""
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


def _draw(d, hq, hkv, prefix, extend, seed, decode=False):
    return W.draw(W.small_spec(batch=len(prefix), hq=hq, hkv=hkv, lq=d, lv=d, prefix=prefix, extend=extend,
                               seed=seed, decode=decode))


def _prefix_rows(wl):
    """Rows of the pool's prefix keys, in index order."""
    at = torch.cat([torch.arange(int(wl.token_offsets[b]), int(wl.token_offsets[b]) + p)
                    for b, p in enumerate(wl.prefix_lens)])
    return wl.k_rows[at].double(), wl.v_rows[at].double()


class Extend:
    def __init__(self, wl):
        self.wl = wl
        self.k, self.v = wl.pool(DEV)
        self.ke, self.ve = wl.extend_kv(DEV)
        self.q, self.qo, self.ptr, self.idx = (x.to(DEV) for x in (wl.q, wl.qo_indptr, wl.kv_indptr, wl.kv_indices))

    def run(self, window, first, cap=0.0, sinks=None, ws=None, **over):
        o = torch.full_like(self.q, float("nan"))
        lse = torch.full(self.q.shape[:2], float("nan"), device=DEV)
        a = dict(k=self.k, v=self.v, ke=self.ke, ve=self.ve, idx=self.idx)
        a.update(over)
        ws = pkx.extend_attention_fwd_streaming(self.q, a["ke"], a["ve"], o, a["k"], a["v"], self.qo, self.ptr,
                                                a["idx"], window, first, self.wl.sm_scale, cap, lse, ws, sinks)
        return o, lse, ws


@pytest.mark.parametrize("d,hq,hkv,prefix,extend,window,first,cap,sinks", [
    (128, 32, 8, [0, 5, 300, 1000], [1, 40, 77, 130], 64, 4, 0.0, False),
    (128, 28, 4, [600, 0, 90, 3000], [200, 1, 19, 5], 100, 1, 20.0, False),
    (64, 12, 3, [0, 999, 45], [500, 2, 129], 33, 128, 0.0, True),    # first tokens end on a tile's border
    (64, 8, 8, [40, 1300], [700, 33], 128, 127, 0.0, False),
    (128, 16, 4, [700, 60], [300, 900], 128, 129, 0.0, True),        # a window start inside the extend keys
    (64, 8, 2, [10, 2000], [1100, 64], 7, 300, 0.0, False),          # more first tokens than prefix
    (128, 8, 2, [500, 0], [9, 257], 1, 0, 0.0, False),               # no first tokens: the plain window
    (128, 8, 1, [4000], [3], 5000, 64, 0.0, False),                  # a window longer than the keys
    (64, 64, 1, [3000, 17], [70, 1], 256, 5, 5.0, True),
    (128, 128, 1, [900], [40], 31, 200, 0.0, False),                 # one token a query tile
    (128, 4, 4, [6000], [1], 17, 2, 0.0, False),                     # split keys of a single row
    (64, 6, 2, [300, 301], [5, 6], 20, 100000, 0.0, False),          # first tokens past all keys
])
def test_extend(d, hq, hkv, prefix, extend, window, first, cap, sinks):
    c = Extend(_draw(d, hq, hkv, prefix, extend, seed=sum(prefix) + d))
    sk = torch.randn(hq, generator=torch.Generator().manual_seed(hq)) * 2 if sinks else None
    o, lse, ws = c.run(window, first, cap, sk.to(DEV) if sinks else None)
    ref = R.extend(c.wl, *_prefix_rows(c.wl), c.ke.cpu(), c.ve.cpu(), window, first, cap, sk)
    R.check(o, lse, ref, d, c.wl.sm_scale, BF16_STEP, tanh_step=TANH_STEP if cap else 0.0)
    assert pkx.workspace_status(ws) == 0


def test_extend_without_window_or_first_is_the_plain_call():
    """first_tokens without a window, and a window without first tokens, give
    the plain call's bits."""
    c = Extend(_draw(128, 16, 4, [300, 0, 77], [40, 200, 1], seed=3))
    for window, first in ((-1, 64), (50, 0)):
        o, lse, _ = c.run(window, first)
        o2, l2 = torch.empty_like(o), torch.empty_like(lse)
        pkx.extend_attention_fwd(c.q, c.ke, c.ve, o2, c.k, c.v, c.qo, c.ptr, c.idx, c.wl.sm_scale, 0.0, window, l2)
        assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_window_and_first_tokens_of_any_size():
    """Past the C int range, and at its limit, they mean all keys."""
    c = Extend(_draw(128, 8, 2, [300, 5], [40, 2], seed=8))
    want, wl_, _ = c.run(-1, 0)
    ref = R.extend(c.wl, *_prefix_rows(c.wl), c.ke.cpu(), c.ve.cpu())
    R.check(want, wl_, ref, 128, c.wl.sm_scale, BF16_STEP)
    for window, first in ((2 ** 32 + 5, 0), (2 ** 31 - 1, 2 ** 31 - 1), (7, 2 ** 40), (-2 ** 40, 3)):
        o, lse, ws = c.run(window, first)
        R.check(o, lse, ref, 128, c.wl.sm_scale, BF16_STEP, f"{window} {first}")
        assert pkx.workspace_status(ws) == 0


def test_extend_reads_nothing_in_the_gap():
    """Keys between the first tokens and every window may hold NaN or bad
    slots; the first tokens and the window may not."""
    c = Extend(_draw(64, 8, 2, [2000], [16], seed=4))
    want, wl_, _ = c.run(100, 4)
    idx = c.idx.clone()
    idx[10:1890] = -5
    o, lse, ws = c.run(100, 4, idx=idx)
    assert torch.equal(o, want) and torch.equal(lse, wl_) and pkx.workspace_status(ws) == 0
    idx[2] = -5
    _, _, ws = c.run(100, 4, idx=idx)
    assert pkx.workspace_status(ws) == pkx.PKX_EDEVICE


def test_extend_strided_rows():
    """Extend rows and pools as slices of wider tensors."""
    c = Extend(_draw(128, 8, 2, [130, 9], [20, 150], seed=5))
    want, wl_, _ = c.run(60, 7)
    n, slots = c.ke.shape[0], c.k.shape[0]
    wide = torch.zeros(n, 2, 400, dtype=torch.bfloat16, device=DEV)
    ke, ve = wide[:, :, 8:136], wide[:, :, 200:328]
    ke.copy_(c.ke), ve.copy_(c.ve)
    pool = torch.zeros(slots, 4, 128, dtype=torch.bfloat16, device=DEV)
    k, v = pool[:, 0::2], pool[:, 1::2]
    k.copy_(c.k), v.copy_(c.v)
    o, lse, _ = c.run(60, 7, ke=ke, ve=ve, k=k, v=v)
    assert torch.equal(o, want) and torch.equal(lse, wl_)


def test_extend_graph_and_side_stream():
    c = Extend(_draw(128, 16, 4, [900, 40], [64, 300], seed=6))
    want, wl_, ws = c.run(128, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, lse, _ = c.run(128, 4)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, want) and torch.equal(lse, wl_)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkx.extend_attention_fwd_streaming(c.q, c.ke, c.ve, out, c.k, c.v, c.qo, c.ptr, c.idx, 128, 4, c.wl.sm_scale,
                                           workspace=ws)
    c.q.mul_(-1.0)
    graph.replay()
    neg, _, _ = c.run(128, 4)
    assert torch.equal(out, neg)


# ------------------------------------------------------------------ decode
@pytest.mark.parametrize("d,hq,hkv,lens,window,first,cap", [
    (128, 32, 8, [1, 0, 31, 128, 129, 500, 4000], 100, 4, 0.0),
    (64, 12, 3, [777, 1, 0, 129], 33, 128, 0.0),
    (128, 28, 4, [900, 45, 3000, 2], 257, 130, 20.0),
    (64, 64, 1, [5000, 17], 64, 1, 0.0),
    (128, 8, 2, [20000], 4096, 300, 0.0),
    (128, 4, 4, [300, 301], 20, 100000, 0.0),
    (64, 128, 1, [260, 31], 1, 0, 0.0),
    (128, 40, 2, [65, 64, 63], 1000, 5, 0.0),
])
def test_decode(d, hq, hkv, lens, window, first, cap):
    wl = _draw(d, hq, hkv, lens, [0] * len(lens), seed=sum(lens) + d, decode=True)
    q = torch.randn(len(lens), hq, d, generator=torch.Generator().manual_seed(d)).bfloat16()
    k, v = wl.pool(DEV)
    o = torch.full((len(lens), hq, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((len(lens), hq), float("nan"), device=DEV)
    ws = pkx.decode_attention_fwd_streaming(q.to(DEV), o, k, v, wl.kv_indptr.to(DEV), wl.kv_indices.to(DEV),
                                            window, first, wl.sm_scale, cap, lse)
    out, k0 = [], 0
    for b, t in enumerate(lens):
        ok = R.visible(torch.tensor([t - 1]), t, window, first)
        out.append(R.attend(q[b:b + 1].double(), wl.k_rows[k0:k0 + t].double(), wl.v_rows[k0:k0 + t].double(), ok,
                            wl.sm_scale, cap))
        k0 += t
    R.check(o, lse, [torch.cat(x) for x in zip(*out)], d, wl.sm_scale, BF16_STEP,
            tanh_step=TANH_STEP if cap else 0.0)
    assert pkx.workspace_status(ws) == 0


def test_decode_small_workspace_gives_the_same():
    """The smallest workspace (one key stream a unit)."""
    lens = [3000, 200]
    wl = _draw(128, 16, 4, lens, [0, 0], seed=9, decode=True)
    q = torch.randn(2, 16, 128, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    k, v = wl.pool(DEV)
    outs = []
    for size in (pkx.decode_workspace_size(2, 16, 4, 128, 128), pkx.decode_workspace_min_size(2, 16, 4, 128, 128)):
        o, lse = torch.empty_like(q), torch.empty(2, 16, device=DEV)
        ws = torch.empty(size, dtype=torch.uint8, device=DEV)
        pkx.decode_attention_fwd_streaming(q, o, k, v, wl.kv_indptr.to(DEV), wl.kv_indices.to(DEV), 700, 64,
                                           wl.sm_scale, lse=lse, workspace=ws)
        assert pkx.workspace_status(ws) == 0
        outs.append((o.float(), lse))
    # two orders of the same sums: each output within its bf16 rounding (2^-8)
    # and the rounding of P (2^-8 of a mean of |v|)
    assert (outs[0][1] - outs[1][1]).abs().max() < 1e-4
    assert (outs[0][0] - outs[1][0]).abs().max() <= 2 * 2.0 ** -8 * (outs[0][0].abs().max() + 1.0)
