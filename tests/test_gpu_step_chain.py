"""GPU tests of a decode step's operators together: one step of a paged cache,
captured graphs, other streams, shared workspaces, large pools, a wait that runs
out."""
import pytest
import torch

import step_reference as R
from paged_kv_extend_gb300 import pkx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE, HQ, HKV, D, TOP = 16, 8, 2, 128, 6


class Step:
    """A decode step over a paged cache: the new token's q and k are normalised,
    rotated and written to the cache, its page's bounds follow, pages are
    selected, and the queries attend to them and, sharing their prefixes, to
    all keys."""

    def __init__(self, lens, seed):
        g = torch.Generator().manual_seed(seed)
        self.lens = lens  # with the new token
        pages = [-(-t // PAGE) for t in lens]
        total = sum(pages) + 2
        perm = torch.randperm(total, generator=g)
        self.ptr = torch.tensor([0] + torch.tensor(pages).cumsum(0).tolist(), dtype=torch.int32)
        self.ids = perm[:sum(pages)].to(torch.int32)
        self.last = torch.tensor([t - (p - 1) * PAGE for t, p in zip(lens, pages)], dtype=torch.int32)
        self.k, self.v = (torch.randn(total * PAGE, HKV, D, generator=g).bfloat16() for _ in range(2))
        b = len(lens)
        self.qkv = torch.randn(b, (HQ + 2 * HKV) * D, generator=g).bfloat16()
        angle = torch.rand(64, D // 2, generator=g, dtype=torch.float64) * 6.3
        self.table = torch.cat([angle.cos(), angle.sin()], 1).float()
        self.pos = torch.tensor([t - 1 for t in lens]) % 64
        self.w = (1 + 0.2 * torch.randn(D, generator=g)).bfloat16()
        ends = [int(self.ids[int(self.ptr[i + 1]) - 1]) for i in range(b)]
        self.new_page = torch.tensor(ends, dtype=torch.int32)
        self.loc = self.new_page.long() * PAGE + self.last.long() - 1
        self.box = torch.zeros(total, HKV, 2, D, dtype=torch.bfloat16)
        full = torch.full((sum(pages),), PAGE)
        full[self.ptr[1:].long() - 1] = self.last.long()
        self.box = R.bounds(self.k, self.ids, full, PAGE, self.box)

    def on_gpu(self):
        return {n: t.to(DEV) for n, t in vars(self).items() if torch.is_tensor(t)}

    def split(self, qkv):
        q, k, v = qkv.split([HQ * D, HKV * D, HKV * D], -1)
        return (x.unflatten(-1, (-1, D)) for x in (q, k, v))

    def run(self, t, out, ws):
        q, k, v = self.split(t["qkv"])
        q, k = pkx.qk_norm_rope(q, k, t["pos"], t["table"], q_out=out["q"], k_out=out["k"], q_weight=t["w"],
                                k_weight=t["w"], cache_loc=t["loc"], v=v, k_buffer=t["k"], v_buffer=t["v"])
        pkx.update_page_bounds(t["k"], t["box"], t["new_page"], PAGE, page_lens=t["last"])
        sel, ws["select"] = pkx.select_pages(q, t["box"], t["ptr"], t["ids"], TOP, 1, 1, selected=out["sel"],
                                             workspace=ws.get("select"))
        ws["pages"] = pkx.decode_attention_fwd_pages(q, out["o"], t["k"], t["v"], t["ptr"], t["ids"], t["last"], PAGE,
                                                     sel, lse=out["lse"], workspace=ws.get("pages"))

    def outputs(self):
        b = len(self.lens)
        nan = lambda *s, dtype=torch.bfloat16: torch.full(s, float("nan"), dtype=dtype, device=DEV)
        return dict(q=nan(b, HQ, D), k=nan(b, HKV, D), o=nan(b, HQ, D), lse=nan(b, HQ, dtype=torch.float32),
                    sel=torch.full((b, HKV, TOP), -9, dtype=torch.int32, device=DEV))

    def check(self, t, out):
        """Each stage against the reference on the stage before's outputs."""
        q, k, v = self.split(t["qkv"].cpu())
        for got, x in ((out["q"], q), (out["k"], k)):
            ref, size = R.rope(x, self.w, 1e-6, 0.0, t["pos"].cpu(), self.table, False, None)
            assert ((got.double().cpu() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -16 * size).all()
        kc, vc = self.k.clone(), self.v.clone()
        kc[self.loc], vc[self.loc] = out["k"].cpu(), v
        assert torch.equal(t["k"].cpu(), kc) and torch.equal(t["v"].cpu(), vc)
        box = R.bounds(kc, self.new_page, self.last, PAGE, self.box)
        assert torch.equal(t["box"].cpu(), box)
        q = out["q"].cpu()
        sel = R.select(q, box, self.ptr, self.ids, TOP, 1, 1)
        assert torch.equal(out["sel"].cpu(), sel)
        o, size = (torch.zeros(q.shape, dtype=torch.float64) for _ in range(2))
        lse = torch.zeros(q.shape[:2], dtype=torch.float64)
        for b, n in enumerate(self.lens):
            for h in range(HKV):
                at = [int(self.ids[int(self.ptr[b]) + s]) * PAGE + j for s in sel[b, h].tolist() if s >= 0
                      for j in range(PAGE) if s * PAGE + j < n]
                rows = slice(h * HQ // HKV, (h + 1) * HQ // HKV)
                o[b, rows], lse[b, rows], size[b, rows] = R.attend(
                    q[b, rows].double(), kc[at, h].double(), vc[at, h].double(), D ** -0.5)
        R.check_attention(out["o"], out["lse"], (o, lse, size))


def test_one_step():
    s = Step([300, 17, 1, 160, 33], 1)
    t, out, ws = s.on_gpu(), s.outputs(), {}
    s.run(t, out, ws)
    assert all(pkx.workspace_status(w) == pkx.PKX_OK for w in ws.values())
    s.check(t, out)


def test_a_captured_step_on_another_stream():
    """Two graphs of the same step that share their workspaces, replayed with
    other inputs, an eager call between them; outputs and cache as of the last."""
    s = Step([300, 17, 1, 160, 33], 2)
    t, out, ws = s.on_gpu(), s.outputs(), {}
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        s.run(t, out, ws)  # warm-up: workspaces, attributes
    stream.synchronize()
    out2 = s.outputs()
    graphs = []
    for o in (out, out2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            s.run(t, o, ws)
        graphs.append(g)
    for seed in (3, 4):
        fresh = Step([300, 17, 1, 160, 33], seed)
        for n, x in fresh.on_gpu().items():
            t[n].copy_(x)
        torch.cuda.synchronize()
        graphs[0].replay()
        torch.cuda.synchronize()
        fresh.check(t, out)
        for x in out2.values():
            x.fill_(-5)
        graphs[1].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        fresh.check(t, out2)
        s.run(t, fresh_out := s.outputs(), ws)
        torch.cuda.synchronize()
        fresh.check(t, fresh_out)


def _paged_all(s, t):
    """Token lists of all keys, for the calls that read every key."""
    return pkx.expand_paged_kv_indices(t["ptr"], t["ids"], t["last"], PAGE, capacity=sum(s.lens))


def test_workspace_shared_with_other_calls():
    """A call's status is its own, whichever call used the workspace before."""
    s = Step([300, 17, 1, 160, 33], 5)
    t, out = s.on_gpu(), s.outputs()
    q = torch.randn(5, HQ, D, device=DEV).bfloat16()
    ptr, idx = _paged_all(s, t)
    o, o2 = torch.empty_like(q), torch.empty_like(q)
    size = max(pkx.decode_workspace_size(5, HQ, HKV, D, D), pkx.decode_shared_workspace_size(5, 1, HQ, HKV, D, D),
               pkx.decode_pages_workspace_size(5, HQ, HKV, D, D, PAGE, 64),
               pkx.select_pages_workspace_size(5, HKV, len(s.ids)))
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    bad_sel = torch.full((5, HKV, TOP), 99, dtype=torch.int32, device=DEV)
    groups = torch.tensor([0, 2], dtype=torch.int32, device=DEV), torch.tensor([0], dtype=torch.int32, device=DEV)
    calls = {
        "decode": lambda: pkx.decode_attention_fwd(q, o, t["k"], t["v"], ptr, idx, workspace=ws),
        "pages": lambda: pkx.decode_attention_fwd_pages(q, o2, t["k"], t["v"], t["ptr"], t["ids"], t["last"], PAGE,
                                                        out["sel"], workspace=ws),
        "many pages": lambda: pkx.decode_attention_fwd_pages(
            q, o2, t["k"], t["v"], t["ptr"], t["ids"], t["last"], PAGE,
            torch.arange(64, dtype=torch.int32, device=DEV).expand(5, HKV, 64).contiguous().clamp(max=0), workspace=ws),
        "select": lambda: pkx.select_pages(q, t["box"], t["ptr"], t["ids"], TOP, selected=out["sel"], workspace=ws),
        "shared": lambda: pkx.decode_attention_fwd_shared(q, o2, t["k"], t["v"], ptr, idx, *groups, workspace=ws),
    }
    calls["select"]()
    broken = lambda: pkx.decode_attention_fwd_pages(q, o2, t["k"], t["v"], t["ptr"], t["ids"], t["last"], PAGE, bad_sel,
                                                    workspace=ws)
    for name, call in calls.items():
        broken()
        assert pkx.workspace_status(ws) == pkx.PKX_EDEVICE
        call()
        assert pkx.workspace_status(ws) == pkx.PKX_OK, name
    calls["decode"]()
    calls["shared"]()
    assert (o.float() - o2.float()).abs().max() <= 2.0 ** -6 * o.float().abs().max()


def test_pools_past_32_bit_offsets():
    """Slots whose elements lie past 2^31 (K) and 2^32 (V, wider strides)."""
    slots, hkv, d = (1 << 21) + 4096, 8, 128
    k = torch.zeros(slots, hkv, d, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros(slots, 2, hkv, d, dtype=torch.bfloat16, device=DEV)[:, 1]
    g = torch.Generator().manual_seed(3)
    n, page = 2048, 64
    first = slots - n  # a multiple of 64
    kk, vv = (torch.randn(n, hkv, d, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(2, 8, d, generator=g).bfloat16()
    loc = torch.arange(first, slots, device=DEV)
    pkx.qk_norm_rope(kk.to(DEV), kk.to(DEV), cache_loc=loc, v=vv.to(DEV), k_buffer=k, v_buffer=v)
    assert torch.equal(k[first:].cpu(), kk) and torch.equal(v[first:].cpu(), vv)
    pages = torch.arange(first // page, slots // page, dtype=torch.int32)
    box = torch.zeros(slots // page, hkv, 2, d, dtype=torch.bfloat16, device=DEV)
    pkx.update_page_bounds(k, box, pages.to(DEV), page)
    assert torch.equal(box[pages.long().to(DEV), :, 1].cpu(), kk.unflatten(0, (-1, page)).amax(1))
    ptr = torch.tensor([0, len(pages), len(pages)], dtype=torch.int32)
    last = torch.tensor([page, 0], dtype=torch.int32)
    on = [x.to(DEV) for x in (q, ptr, pages, last)]
    sel, ws = pkx.select_pages(on[0], box, on[1], on[2], 8)
    ref_sel = R.select(q, box[pages.long().to(DEV)].cpu(), ptr, torch.arange(len(pages)), 8, 1, 1)
    assert torch.equal(sel.cpu(), ref_sel)
    o, lse = torch.empty_like(on[0]), torch.empty(2, 8, device=DEV)
    ref = [torch.zeros(2, 8, d, dtype=torch.float64), torch.full((2, 8), float("-inf"), dtype=torch.float64),
           torch.zeros(2, 8, d, dtype=torch.float64)]
    pkx.decode_attention_fwd_pages(on[0], o, k, v, on[1], on[2], on[3], page, sel, lse=lse)
    for h in range(hkv):
        at = torch.cat([torch.arange(s * page, (s + 1) * page) for s in ref_sel[0, h].tolist()])
        for r, x in zip(ref, R.attend(q[0, h:h + 1].double(), kk[at, h].double(), vv[at, h].double(), d ** -0.5)):
            r[0, h:h + 1] = x
    R.check_attention(o, lse, ref)
    # both sequences over all keys: their prefix shared
    members = 40
    q = torch.randn(members, 8, d, generator=g).bfloat16()
    idx = torch.arange(first, slots, dtype=torch.int32).repeat(members)
    ptr = torch.arange(members + 1, dtype=torch.int32) * n
    o, lse = torch.empty(members, 8, d, dtype=torch.bfloat16, device=DEV), torch.empty(members, 8, device=DEV)
    ws = pkx.decode_attention_fwd_shared(q.to(DEV), o, k, v, ptr.to(DEV), idx.to(DEV),
                                         torch.tensor([0, members], dtype=torch.int32, device=DEV),
                                         torch.tensor([n - 100], dtype=torch.int32, device=DEV), lse=lse)
    assert pkx.workspace_status(ws) == pkx.PKX_OK and int(ws.view(torch.int32)[1]) > 0
    ref = [torch.zeros(members, 8, d, dtype=torch.float64), torch.zeros(members, 8, dtype=torch.float64),
           torch.zeros(members, 8, d, dtype=torch.float64)]
    for h in range(hkv):
        for r, x in zip(ref, R.attend(q[:, h].double(), kk[:, h].double(), vv[:, h].double(), d ** -0.5)):
            r[:, h] = x
    R.check_attention(o, lse, ref)


def test_a_wait_that_runs_out():
    """The stall hook stops the prefix units' softmax: the call reports it, and
    the next one is clean."""
    n, members = 3000, 20
    k, v = (torch.randn(n + 100, 8, 128, device=DEV).bfloat16() for _ in range(2))
    q = torch.randn(members, 32, 128, device=DEV).bfloat16()
    idx = torch.arange(n, dtype=torch.int32, device=DEV).repeat(members)
    ptr = torch.arange(members + 1, dtype=torch.int32, device=DEV) * n
    groups = (torch.tensor([0, members], dtype=torch.int32, device=DEV), torch.tensor([n], dtype=torch.int32, device=DEV))
    o, want = torch.empty_like(q), torch.empty_like(q)
    run = lambda out: pkx.decode_attention_fwd_shared(q, out, k, v, ptr, idx, *groups)
    assert pkx.workspace_status(run(want)) == pkx.PKX_OK
    pkx.set_wait_limit_ns(3_000_000)
    pkx.set_stall_injection(True)
    try:
        status = pkx.workspace_status(run(o))
    finally:
        pkx.set_stall_injection(False)
        pkx.set_wait_limit_ns(0)
    assert status == pkx.PKX_ETIMEOUT
    assert pkx.workspace_status(run(o)) == pkx.PKX_OK
    assert torch.equal(o, want)


def test_bindings_check_shapes_on_the_gpu():
    bf, i32 = torch.bfloat16, torch.int32
    z = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype, device=DEV)
    q, k, table = z(3, 4, 64), z(16, 2, 64), z(10, 64, dtype=torch.float32)
    pos, loc = z(3, dtype=torch.int64), z(3, dtype=torch.int64)
    kn = z(3, 2, 64)
    bad = [
        lambda: pkx.qk_norm_rope(q, z(2, 2, 64)), lambda: pkx.qk_norm_rope(q, z(3, 2, 32)),
        lambda: pkx.qk_norm_rope(q, kn, pos), lambda: pkx.qk_norm_rope(q, kn, None, table),
        lambda: pkx.qk_norm_rope(q, kn, pos[:2], table), lambda: pkx.qk_norm_rope(q, kn, pos.int(), table),
        lambda: pkx.qk_norm_rope(q, kn, pos, table.double()), lambda: pkx.qk_norm_rope(q, kn, q_weight=z(32)),
        lambda: pkx.qk_norm_rope(q, kn, pos, table, pair_axis=z(31, dtype=torch.uint8)),
        lambda: pkx.qk_norm_rope(q, kn, v=kn), lambda: pkx.qk_norm_rope(q, kn, cache_loc=loc),
        lambda: pkx.qk_norm_rope(q, kn, cache_loc=loc, k_buffer=k, v=kn),
        lambda: pkx.qk_norm_rope(q, kn, cache_loc=loc[:2], k_buffer=k),
        lambda: pkx.qk_norm_rope(q, kn, cache_loc=loc, k_buffer=z(16, 3, 64)),
        lambda: pkx.qk_norm_rope(q, kn, cache_loc=loc, k_buffer=k, v=kn, v_buffer=z(15, 2, 64)),
        lambda: pkx.qk_norm_rope(q, kn, q_out=z(3, 4, 32)), lambda: pkx.qk_norm_rope(q.float(), kn),
        lambda: pkx.update_page_bounds(k, z(3, 2, 2, 64), z(1, dtype=i32), 8),
        lambda: pkx.update_page_bounds(k, z(2, 2, 2, 32), z(1, dtype=i32), 8),
        lambda: pkx.update_page_bounds(k, z(2, 2, 2, 64), z(1, dtype=i32), 0),
        lambda: pkx.update_page_bounds(k, z(2, 2, 2, 64), z(2, dtype=i32), 8, page_lens=z(1, dtype=i32)),
        lambda: pkx.select_pages(q, z(2, 2, 2, 32), z(4, dtype=i32), z(2, dtype=i32), 2),
        lambda: pkx.select_pages(q, z(2, 2, 2, 64), z(3, dtype=i32), z(2, dtype=i32), 2),
        lambda: pkx.select_pages(q, z(2, 2, 2, 64), z(4, dtype=i32), z(2, dtype=i32), 2, selected=z(3, 2, 3, dtype=i32)),
        lambda: pkx.decode_attention_fwd_pages(q, q, k, k, z(4, dtype=i32), z(1, dtype=i32), z(2, dtype=i32), 8,
                                               z(3, 2, 2, dtype=i32)),
        lambda: pkx.decode_attention_fwd_pages(q, q, k, k, z(4, dtype=i32), z(1, dtype=i32), z(3, dtype=i32), 8,
                                               z(3, 1, 2, dtype=i32)),
        lambda: pkx.decode_attention_fwd_shared(q, q, k, z(15, 2, 64), z(4, dtype=i32), z(1, dtype=i32),
                                                z(2, dtype=i32), z(1, dtype=i32)),
        lambda: pkx.decode_attention_fwd_shared(q, q, k, k, z(4, dtype=i32), z(1, dtype=i32), z(2, dtype=i32),
                                                z(2, dtype=i32)),
        lambda: pkx.decode_attention_fwd_shared(q, z(3, 4, 32), k, k, z(4, dtype=i32), z(1, dtype=i32),
                                                z(2, dtype=i32), z(1, dtype=i32)),
        lambda: pkx.decode_attention_fwd_shared(z(3, 4, 32), q, k, k, z(4, dtype=i32), z(1, dtype=i32),
                                                z(2, dtype=i32), z(1, dtype=i32)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    with pytest.raises(pkx.PkxError):
        pkx.qk_norm_rope(q, kn, torch.zeros(2, 3, dtype=torch.int64, device=DEV), table)  # axes without pair_axis
    with pytest.raises(pkx.PkxError):
        pkx.select_pages(q, z(2, 2, 2, 64), z(4, dtype=i32), z(2, dtype=i32), 0)
