"""Cases that measure a decode step's operators around a paged KV pool.

Operators (entry points of ``paged_kv_extend_gb300.pkx``):
  qk_norm_rope                  per-head RMS norm and position rotation of
                                queries and keys, with the KV write
  update_page_bounds            smallest and largest key value of each page
  select_pages                  the pages whose bounds promise the largest logits
  decode_attention_fwd_pages    decode attention over the selected pages
  decode_attention_fwd_shared   decode attention for sequences in groups that
                                share a prefix, whose keys are read once

The rotation.  Pair i of a row's first ``rotary`` dims is (x[i], x[i + r / 2]),
or (x[2i], x[2i + 1]) where ``interleaved``; it becomes (a c - b s, b c + a s)
with c = table[p, i] and s = table[p, r / 2 + i], p being the token's position
on the pair's axis (one axis for text; time, height and width for video).

The page score of (sequence, KV head, page).  With qp[d] the sum over the
group's query heads, in order, of max(q, 0) and qn[d] that of min(q, 0), and
lo / hi the page's bounds, it is tree(qn * lo) + tree(qp * hi), where tree()
adds neighbours pairwise (0 + 1, 2 + 3, ..., then the sums likewise) and every
product and sum is rounded to fp32.  A sequence of at most ``top_k`` pages
takes all of them; otherwise its first and last pages and the others by score,
equal scores by the lower page.

``run`` computes the operators in plain torch, or, where ``own`` is true,
calls the framework.
"""
import random

import torch

own = False

DEV = "cuda"
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's new tokens of 64 running sequences, written to the cache
        dict(name="rope_decode_step", op="rope", tokens=64, hq=32, hkv=8, d=128, rotary=128,
             norm=True, interleaved=False, axes=1, kv="bf16"),
        # a prefill chunk, normalised, rotated and written in one pass
        dict(name="rope_prefill", op="rope", tokens=16384, hq=32, hkv=8, d=128, rotary=128,
             norm=True, interleaved=False, axes=1, kv="bf16"),
        # frames of a video with three axes, neighbouring pairs, half of the dims rotated, fp8 cache
        dict(name="rope_video", op="rope", tokens=5001, hq=28, hkv=4, d=128, rotary=64,
             norm=False, interleaved=True, axes=3, kv="e4m3"),
        # after a decode step: the page that each of 64 sequences writes to
        dict(name="bounds_decode_step", op="bounds", pages=64, page=64, hkv=8, d=128, kv="bf16",
             ragged=1),
        # after a long prompt: all of its pages
        dict(name="bounds_prompt", op="bounds", pages=2048, page=64, hkv=8, d=128, kv="bf16",
             ragged=0),
        # a few short chats, one just begun, one slot of padding
        dict(name="pages_short", op="pages", batch=5, hq=12, hkv=3, d=64, keys=777, page=16,
             top=9, first=1, last=2, ragged=3, kv="bf16"),
        # the serving step at 32768 cached tokens, a sixteenth of the cache read
        dict(name="pages_batch", op="pages", batch=64, hq=32, hkv=8, d=128, keys=32768, page=64,
             top=32, first=1, last=2, ragged=0, kv="bf16"),
        # one user with a very long document in an fp8 cache
        dict(name="pages_single_long", op="pages", batch=1, hq=28, hkv=4, d=128, keys=131071,
             page=32, top=128, first=2, last=4, ragged=0, kv="e4m3"),
        # a few chats that begin with the same lines
        dict(name="shared_short", op="shared", groups=1, size=5, alone=1, hq=12, hkv=3, d=64,
             prefix=201, keys=33, ragged=5, kv="bf16"),
        # a system prompt of 8192 tokens that 64 conversations share
        dict(name="shared_system_prompt", op="shared", groups=1, size=64, alone=0, hq=32, hkv=8,
             d=128, prefix=8192, keys=1024, ragged=7, kv="bf16"),
        # parallel samples: eight prompts, eight continuations each, fp8 cache
        dict(name="shared_samples", op="shared", groups=8, size=8, alone=3, hq=28, hkv=4, d=128,
             prefix=4096, keys=500, ragged=9, kv="e4m3"),
        # questions to one long document
        dict(name="shared_document", op="shared", groups=1, size=256, alone=0, hq=32, hkv=8, d=128,
             prefix=32768, keys=64, ragged=11, kv="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["rope", "rope", "bounds", "pages", "pages", "shared", "shared"])
    d = rng.choice([64, 128])
    kv = rng.choice(["bf16", "bf16", "e4m3", "e5m2"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 4] if hkv == 8 else [1, 4, 7, 8])
    if op == "rope":
        return dict(op=op, tokens=_log(rng, 1, 16384), hq=hq, hkv=hkv, d=d,
                    rotary=rng.choice([d, d // 2, 32]), norm=rng.random() < 0.6,
                    interleaved=rng.random() < 0.4, axes=rng.choice([1, 1, 2, 3]), kv=kv)
    if op == "bounds":
        return dict(op=op, pages=_log(rng, 1, 2048), page=rng.choice([16, 32, 64]), hkv=hkv, d=d,
                    kv=kv, ragged=rng.choice([0, rng.randint(1, 1 << 20)]))
    if op == "pages":
        return dict(op=op, batch=_log(rng, 1, 48), hq=hq, hkv=hkv, d=d, keys=_log(rng, 1, 32768),
                    page=rng.choice([16, 32, 64]), top=_log(rng, 4, 32), first=rng.randint(0, 2),
                    last=rng.randint(1, 2), ragged=rng.choice([0, rng.randint(1, 1 << 20)]), kv=kv)
    groups = _log(rng, 1, 8)
    return dict(op=op, groups=groups, size=_log(rng, 1, 96 // groups), alone=rng.randint(0, 3),
                hq=hq, hkv=hkv, d=d, prefix=_log(rng, 1, 16384), keys=_log(rng, 1, 1000),
                ragged=rng.choice([0, rng.randint(1, 1 << 20)]), kv=kv)


def _page_lens(case):
    """Keys in each listed page; a ragged case fills them partly."""
    r = random.Random(case["ragged"])
    return [case["page"] if not case["ragged"] else r.randint(1, case["page"])
            for _ in range(case["pages"])]


def _seq_lens(case):
    """Cached keys of each sequence of a "pages" case.  Ragged batches hold a
    sequence of one key and an empty one."""
    r = random.Random(case["ragged"])
    lens = [case["keys"] if not case["ragged"] else r.randint(1, case["keys"])
            for _ in range(case["batch"])]
    if case["ragged"] and len(lens) >= 3:
        lens[1], lens[2] = 1, 0
    return lens


def _groups(case):
    """(shared keys, own keys of each member) of each group; the sequences that
    stand alone come last as groups of one without shared keys."""
    r = random.Random(case["ragged"])
    rag = case["ragged"]
    out = []
    for _ in range(case["groups"]):
        p = case["prefix"] if not rag or case["groups"] == 1 else r.randint(1, case["prefix"])
        out.append((p, [case["keys"] if not rag else r.randint(0, case["keys"])
                        for _ in range(case["size"])]))
    for i in range(case["alone"]):
        out.append((0, [0 if i == 1 else r.randint(1, case["prefix"])]))
    return out


def work(case):
    op, hkv, d = case["op"], case["hkv"], case["d"]
    if op == "rope":
        n, hq, kv = case["tokens"], case["hq"], 2 if case["kv"] == "bf16" else 1
        row = 2 * hq * d * 2 + 2 * hkv * d * 2 + hkv * d * (2 + 2 * kv)  # q, k in and out; v; pool
        return {"bytes": n * (row + 8 * case["axes"] + 8) + 4 * min(n * case["axes"], 32768) * case["rotary"],
                "flops": n * (hq + hkv) * (3 * case["rotary"] + (4 * d if case["norm"] else 0))}
    size = 2 if case["kv"] == "bf16" else 1
    if op == "bounds":
        keys = sum(_page_lens(case))
        return {"bytes": keys * hkv * d * size + case["pages"] * (hkv * d * 4 + 8),
                "flops": 2 * keys * hkv * d}
    hq = case["hq"]
    if op == "pages":
        lens = _seq_lens(case)
        pages = [-(-t // case["page"]) for t in lens]
        keys = sum(min(t, case["top"] * case["page"]) for t in lens)
        scored = sum(p for p in pages if p > case["top"])
        return {"bytes": hkv * (scored * d * 4 + keys * d * 2 * size + 4 * len(lens) * case["top"])
                + 4 * sum(pages) + len(lens) * hq * (4 * d + 4),
                "flops": 4 * keys * hq * d + 4 * scored * hkv * d}
    groups = _groups(case)
    batch = sum(len(o) for _, o in groups)
    read = sum(p + sum(o) for p, o in groups)
    pairs = sum(len(o) * p + sum(o) for p, o in groups)
    return {"bytes": read * (hkv * d * 2 * size + 4) + batch * hq * (4 * d + 4),
            "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ inputs
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _pool(g, slots, hkv, d, kv):
    """A filled pool; keys of neighbouring slots are alike, as a text's are."""
    out = torch.empty(slots, hkv, d, dtype=torch.bfloat16 if kv == "bf16" else FP8[kv][0], device=DEV)
    step = max(64, (1 << 28) // (hkv * d) // 64 * 64)
    for s in range(0, slots, step):
        e = min(slots, s + step)
        x = _normal(g, e - s, hkv, d)
        topic = _normal(g, -(-(e - s) // 64), hkv, d).repeat_interleave(64, 0)[:e - s]
        out[s:e] = (x * 0.8 + topic * 0.6).to(out.dtype)
    return out


def _scales(case):
    return (1.0, 1.0) if case["kv"] == "bf16" else (0.75, 1.5)


def _cumsum0(lens):
    return torch.tensor([0] + torch.tensor(lens, dtype=torch.int64).cumsum(0).tolist(),
                        dtype=torch.int32, device=DEV)


def _rope_table(positions, rotary):
    """cos and sin of each pair's angle, fp32 [positions, rotary]."""
    freq = 10000.0 ** (-torch.arange(rotary // 2, dtype=torch.float64, device=DEV) * 2 / rotary)
    angle = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _prepare_rope(case, g):
    n, hq, hkv, d, axes = (case[k] for k in ("tokens", "hq", "hkv", "d", "axes"))
    qkv = _normal(g, n, (hq + 2 * hkv) * d)  # one projection's output
    q, k, v = qkv.split([hq * d, hkv * d, hkv * d], -1)
    slots = n + n // 4 + 3
    dt = torch.bfloat16 if case["kv"] == "bf16" else FP8[case["kv"]][0]
    st = dict(q=q.view(n, hq, d), k=k.view(n, hkv, d), v=v.view(n, hkv, d),
              table=_rope_table(32768, case["rotary"]),
              loc=torch.randperm(slots, generator=g, device=DEV)[:n],
              kc=torch.zeros(slots, hkv, d, device=DEV).to(dt),
              vc=torch.zeros(slots, hkv, d, device=DEV).to(dt), qw=None, kw=None, axis=None)
    shape = (n,) if axes == 1 else (axes, n)
    st["pos"] = torch.randint(0, 32768, shape, generator=g, device=DEV)
    if axes > 1:  # time, height, width: a quarter, and equal shares of the rest
        half = case["rotary"] // 2
        cut = half // 4
        st["axis"] = torch.tensor([0 if i < cut else 1 + (i - cut) * (axes - 1) // (half - cut)
                                   for i in range(half)], dtype=torch.uint8, device=DEV)
    if case["norm"]:
        st["qw"] = (1 + 0.2 * _normal(g, d)).bfloat16()
        st["kw"] = (1 + 0.2 * _normal(g, d)).bfloat16()
    return st


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, d, hkv, kv = case["op"], case["d"], case["hkv"], case["kv"]
    if op == "rope":
        return dict(case=case, **_prepare_rope(case, g))
    ks, vs = _scales(case)
    st = dict(case=case, ks=ks, vs=vs, ws=None, ws2=None, scale=d ** -0.5)
    if op == "bounds":
        n = case["pages"]
        total = n + n // 8 + 1
        st["k"] = _pool(g, total * case["page"], hkv, d, kv)
        st["ids"] = torch.randperm(total, generator=g, device=DEV)[:n].to(torch.int32)
        st["lens"] = torch.tensor(_page_lens(case), dtype=torch.int32, device=DEV)
        st["bounds"] = torch.zeros(total, hkv, 2, d, dtype=torch.bfloat16, device=DEV)
        return st
    if op == "pages":
        lens, page = _seq_lens(case), case["page"]
        pages = [-(-t // page) for t in lens]
        total = sum(pages) + 2
        st.update(lens=lens, pages=pages, indptr=_cumsum0(pages),
                  ids=torch.randperm(total, generator=g, device=DEV)[:sum(pages)].to(torch.int32),
                  last=torch.tensor([t - (p - 1) * page if p else 0 for t, p in zip(lens, pages)],
                                    dtype=torch.int32, device=DEV),
                  k=_pool(g, total * page, hkv, d, kv), v=_pool(g, total * page, hkv, d, kv))
        # (the rows behind a sequence's last key count as keys here: wider
        # bounds, as a page that was used before leaves them)
        st["bounds"] = torch.empty(total, hkv, 2, d, dtype=torch.bfloat16, device=DEV)
        step = max(1, (1 << 28) // (page * hkv * d))
        for s in range(0, total, step):
            x = st["k"][s * page:(s + step) * page].bfloat16().view(-1, page, hkv, d)
            st["bounds"][s:s + step, :, 0], st["bounds"][s:s + step, :, 1] = x.amin(1), x.amax(1)
        st["q"] = _normal(g, len(lens), case["hq"], d)
        return st
    groups = _groups(case)
    n_idx = sum(p + sum(o) for p, o in groups)
    slots = n_idx + n_idx // 4 + 16
    free = torch.randperm(slots, generator=g, device=DEV)[:n_idx].to(torch.int32)
    parts, lens, at = [], [], 0
    for p, own_keys in groups:
        prefix, at = free[at:at + p], at + p
        for t in own_keys:
            parts += [prefix, free[at:at + t]]
            lens.append(p + t)
            at += t
    n = case["groups"]
    st.update(groups=groups, lens=lens, indptr=_cumsum0(lens), idx=torch.cat(parts),
              group_indptr=_cumsum0([case["size"]] * n),
              shared=torch.tensor([p for p, _ in groups[:n]], dtype=torch.int32, device=DEV),
              k=_pool(g, slots, hkv, d, kv), v=_pool(g, slots, hkv, d, kv),
              q=_normal(g, len(lens), case["hq"], d))
    return st


# -------------------------------------------------------------- plain form
def _to_pool(x, kv):
    """A row as the pool holds it (the scales here are 1)."""
    if kv == "bf16":
        return x
    dt, top = FP8[kv]
    return x.float().clamp(-top, top).to(dt)


def _rows_at(pool, at):
    """Rows of a pool (one-byte types are indexed as bytes)."""
    if pool.dtype == torch.bfloat16:
        return pool[at]
    return pool.view(torch.uint8)[at].view(pool.dtype)


def _plain_rope(st):
    case = st["case"]
    r, half = case["rotary"], case["rotary"] // 2
    pos = st["pos"] if st["pos"].dim() == 2 else st["pos"][None]
    axis = st["axis"].long() if st["axis"] is not None else torch.zeros(half, dtype=torch.int64, device=DEV)
    at = pos[axis].T  # [n, half]: the position of each pair
    i = torch.arange(half, device=DEV)
    c, s = st["table"][at, i][:, None], st["table"][at, half + i][:, None]

    def turn(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
        rot, rest = y[..., :r], y[..., r:]
        if case["interleaved"]:
            a, b = rot[..., 0::2], rot[..., 1::2]
            rot = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
        else:
            a, b = rot[..., :half], rot[..., half:]
            rot = torch.cat([a * c - b * s, b * c + a * s], -1)
        return torch.cat([rot, rest], -1).bfloat16()

    q, k = turn(st["q"], st["qw"]), turn(st["k"], st["kw"])
    for pool, x in ((st["kc"], k), (st["vc"], st["v"])):
        x = _to_pool(x, case["kv"])
        if case["kv"] == "bf16":
            pool[st["loc"]] = x
        else:
            pool.view(torch.uint8)[st["loc"]] = x.view(torch.uint8)
    return q, k, st["kc"], st["vc"]


def _plain_bounds(st):
    case = st["case"]
    page = case["page"]
    ids = st["ids"].long()
    x = _rows_at(st["k"].unflatten(0, (-1, page)), ids).float()
    have = torch.arange(page, device=DEV)[None, :] < st["lens"][:, None]
    have = have[:, :, None, None]
    st["bounds"][ids, :, 0] = torch.where(have, x, float("inf")).amin(1).bfloat16()
    st["bounds"][ids, :, 1] = torch.where(have, x, float("-inf")).amax(1).bfloat16()
    return st["bounds"]


def _tree(x):
    while x.shape[-1] > 1:
        x = x[..., 0::2] + x[..., 1::2]
    return x[..., 0]


def _plain_select(st):
    case = st["case"]
    hkv, top, first, last = case["hkv"], case["top"], case["first"], case["last"]
    out = torch.full((len(st["lens"]), hkv, top), -1, dtype=torch.int32, device=DEV)
    q = st["q"].float().unflatten(1, (hkv, -1))
    qp, qn = torch.zeros_like(q[:, :, 0]), torch.zeros_like(q[:, :, 0])
    for i in range(q.shape[2]):
        qp = qp + q[:, :, i].clamp(min=0)
        qn = qn + q[:, :, i].clamp(max=0)
    at = 0
    for b, n in enumerate(st["pages"]):
        if n <= top:
            out[b, :, :n] = torch.arange(n, device=DEV)
        else:
            x = st["bounds"][st["ids"][at:at + n].long()].float()
            score = (_tree(x[:, :, 0] * qn[b]) + _tree(x[:, :, 1] * qp[b])).T  # [hkv, n]
            order = torch.sort(score[:, first:n - last], dim=-1, descending=True, stable=True).indices
            always = torch.cat([torch.arange(first, device=DEV), torch.arange(n - last, n, device=DEV)])
            pick = torch.cat([order[:, :top - first - last] + first, always.expand(hkv, -1)], 1)
            out[b] = pick.sort(-1).values
        at += n
    return out


def _softmax_parts(parts):
    """Softmax over the concatenation of score tensors, by part, and the log sum."""
    m = torch.cat([p.amax(-1, keepdim=True) for p in parts if p.shape[-1]], -1).amax(-1, keepdim=True)
    m0 = torch.where(m == float("-inf"), 0.0, m)
    e = [(p - m0).exp() for p in parts]
    z = sum(p.sum(-1, keepdim=True) for p in e)
    return [p / torch.where(z > 0, z, 1.0) for p in e], (m + z.log()).squeeze(-1)


def _plain_pages(st):
    case = st["case"]
    sel = _plain_select(st)
    page, hkv = case["page"], case["hkv"]
    q = st["q"].float().unflatten(1, (hkv, -1))  # [b, hkv, g, d]
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], device=DEV)
    step = max(1, (1 << 29) // (hkv * case["top"] * page * case["d"]))
    heads = torch.arange(hkv, device=DEV)[None, :, None]
    n_pages = torch.tensor(st["pages"], device=DEV)
    for b in range(0, q.shape[0], step):
        s = sel[b:b + step].long()
        n = n_pages[b:b + step, None, None]
        have = (s >= 0)[..., None] & ((s < n - 1)[..., None] | (
            torch.arange(page, device=DEV) < st["last"][b:b + step, None, None, None]))
        flat = (st["indptr"][:-1][b:b + step, None, None] + s.clamp(min=0)).clamp(max=max(len(st["ids"]) - 1, 0))
        ids = st["ids"][flat].long() if len(st["ids"]) else torch.zeros_like(flat)
        at = (ids[..., None] * page + torch.arange(page, device=DEV)).flatten(2)
        if case["kv"] == "bf16":
            k, v = st["k"][at, heads].float(), st["v"][at, heads].float()
        else:
            k, v = (st[x].view(torch.uint8)[at, heads].view(st[x].dtype).float() * f
                    for x, f in (("k", st["ks"]), ("v", st["vs"])))
        x = (q[b:b + step] @ k.transpose(-1, -2)) * st["scale"]
        x = x.masked_fill(~have.flatten(2)[:, :, None], float("-inf"))
        (p,), lse[b:b + step] = _softmax_parts([x])
        o[b:b + step] = p @ v
    return sel, o.flatten(1, 2).bfloat16(), lse.flatten(1, 2)


def _plain_shared(st):
    case = st["case"]
    hkv = case["hkv"]
    q = st["q"].float().unflatten(1, (hkv, -1))  # [b, hkv, g, d]
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    rows = lambda x, at: _rows_at(st[x], at.long()).float() * (st["ks"] if x == "k" else st["vs"])
    b = at = 0
    for p, own_keys in st["groups"]:
        n, most = len(own_keys), max(own_keys)
        pre = st["idx"][at:at + p]
        own_idx = torch.zeros(n, most, dtype=torch.int32, device=DEV)
        for i, t in enumerate(own_keys):
            own_idx[i, :t] = st["idx"][at + p:at + p + t]
            at += p + t
        have = torch.arange(most, device=DEV) < torch.tensor(own_keys, device=DEV)[:, None]
        g = q[b:b + n]
        kp, vp = (rows(x, pre).transpose(0, 1) for x in "kv")             # [hkv, p, d]
        ko, vo = (rows(x, own_idx).transpose(1, 2) for x in "kv")         # [n, hkv, most, d]
        flat = g.transpose(0, 1).flatten(1, 2)                            # [hkv, n * g, d]
        x1 = ((flat @ kp.transpose(-1, -2)) * st["scale"]).unflatten(1, (n, -1)).transpose(0, 1)
        x2 = (g @ ko.transpose(-1, -2)) * st["scale"]
        x2 = x2.masked_fill(~have[:, None, None], float("-inf"))
        if p + most == 0:
            o[b:b + n], lse[b:b + n] = 0.0, float("-inf")
        else:
            (p1, p2), lse[b:b + n] = _softmax_parts([x1, x2])
            o1 = (p1.transpose(0, 1).flatten(1, 2) @ vp).unflatten(1, (n, -1)).transpose(0, 1)
            o[b:b + n] = o1 + p2 @ vo
        b += n
    return o.flatten(1, 2).bfloat16(), lse.flatten(1, 2)


# --------------------------------------------------------------------- run
def _own(st):
    from paged_kv_extend_gb300 import pkx
    case = st["case"]
    op = case["op"]
    if op == "rope":
        q, k = pkx.qk_norm_rope(
            st["q"], st["k"], st["pos"], st["table"], q_weight=st["qw"], k_weight=st["kw"], eps=1e-6,
            interleaved=case["interleaved"], pair_axis=st["axis"], cache_loc=st["loc"], v=st["v"],
            k_buffer=st["kc"], v_buffer=st["vc"])
        return q, k, st["kc"], st["vc"]
    if op == "bounds":
        return pkx.update_page_bounds(st["k"], st["bounds"], st["ids"], case["page"], page_lens=st["lens"])
    q = st["q"]
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=DEV)
    scales = dict(k_scale=st["ks"], v_scale=st["vs"])
    if op == "pages":
        sel, st["ws"] = pkx.select_pages(q, st["bounds"], st["indptr"], st["ids"], case["top"],
                                         first_pages=case["first"], last_pages=case["last"],
                                         workspace=st["ws"])
        st["ws2"] = pkx.decode_attention_fwd_pages(
            q, o, st["k"], st["v"], st["indptr"], st["ids"], st["last"], case["page"], sel,
            st["scale"], lse=lse, workspace=st["ws2"], **scales)
        return sel, o, lse
    st["ws"] = pkx.decode_attention_fwd_shared(
        q, o, st["k"], st["v"], st["indptr"], st["idx"], st["group_indptr"], st["shared"],
        st["scale"], lse=lse, workspace=st["ws"], **scales)
    return o, lse


def run(state):
    if own:
        return _own(state)
    plain = {"rope": _plain_rope, "bounds": _plain_bounds, "pages": _plain_pages, "shared": _plain_shared}
    return plain[state["case"]["op"]](state)


# ------------------------------------------------------------------- exact
def _exact_rope(st):
    case = st["case"]
    r = case["rotary"]
    half, n = r // 2, case["tokens"]
    first = [2 * i if case["interleaved"] else i for i in range(half)]
    second = [2 * i + 1 if case["interleaved"] else i + half for i in range(half)]
    outs = []
    for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
        y = x.double()
        if w is not None:
            y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
        out = y.clone()
        for i in range(half):
            p = st["pos"] if st["axis"] is None else st["pos"][int(st["axis"][i])]
            c, s = (st["table"][p, j].double()[:, None] for j in (i, half + i))
            a, b = y[..., first[i]], y[..., second[i]]
            out[..., first[i]] = a * c - b * s
            out[..., second[i]] = a * s + b * c
        outs.append(out)
    pools = []
    for pool, x in ((st["kc"], outs[1]), (st["vc"], st["v"].double())):
        full = torch.zeros(pool.shape, dtype=torch.float64, device=DEV)
        if case["kv"] != "bf16":  # an fp8 pool holds the value nearest to the bf16 row
            dt, top = FP8[case["kv"]]
            x = x.float().bfloat16().double().clamp(-top, top).float().to(dt).double()
        full.index_copy_(0, st["loc"], x)
        pools.append(full)
    return (*outs, *pools)


def _exact_bounds(st):
    case = st["case"]
    out = st["bounds"].double()
    rows = st["k"].double().view(-1, case["page"], case["hkv"], case["d"])
    for i, (p, t) in enumerate(zip(st["ids"].tolist(), st["lens"].tolist())):
        out[p, :, 0], out[p, :, 1] = rows[p, :t].min(0).values, rows[p, :t].max(0).values
    return out


def _fold32(terms):
    """The pairwise sum of the definition: float64 sums rounded to fp32 each."""
    while terms.shape[-1] > 1:
        terms = terms.unflatten(-1, (-1, 2)).sum(-1).float().double()
    return terms.squeeze(-1)


def _exact_select(st):
    case = st["case"]
    hkv, top, first, last = case["hkv"], case["top"], case["first"], case["last"]
    group = case["hq"] // hkv
    out = torch.full((len(st["lens"]), hkv, top), -1, dtype=torch.int32)
    start = st["indptr"].tolist()
    for b, n in enumerate(st["pages"]):
        if n <= top:
            out[b, :, :n] = torch.arange(n)
            continue
        box = st["bounds"][st["ids"][start[b]:start[b] + n].long()].double()
        for h in range(hkv):
            pos = torch.zeros(case["d"], dtype=torch.float64, device=DEV)
            neg = pos.clone()
            for x in st["q"][b, h * group:(h + 1) * group].double():
                pos = (pos + torch.where(x > 0, x, 0.0)).float().double()
                neg = (neg + torch.where(x < 0, x, 0.0)).float().double()
            score = (_fold32((box[:, h, 0] * neg).float().double())
                     + _fold32((box[:, h, 1] * pos).float().double())).float()
            middle = sorted(enumerate(score.tolist()[first:n - last], first), key=lambda e: (-e[1], e[0]))
            pick = [*range(first), *range(n - last, n), *(p for p, _ in middle[:top - first - last])]
            out[b, h] = torch.tensor(sorted(pick))
    return out.to(DEV)


def _exact_rows(st, name, slots, head):
    return _rows_at(st[name][:, head], slots).double() * (st["ks"] if name == "k" else st["vs"])


def _exact_attend(st, q, k, v):
    """q [g, d] over keys k [t, d]: (o, lse)."""
    if not k.shape[0]:
        return torch.zeros_like(q), torch.full((q.shape[0],), float("-inf"), dtype=q.dtype, device=DEV)
    s = (q @ k.T) * st["scale"]
    return torch.softmax(s, -1) @ v, torch.logsumexp(s, -1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(st)
    if case["op"] == "bounds":
        return _exact_bounds(st)
    group, hkv = case["hq"] // case["hkv"], case["hkv"]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device=DEV)
    sel = _exact_select(st) if case["op"] == "pages" else None
    start = st["indptr"].tolist()
    for b, t in enumerate(st["lens"]):
        for h in range(hkv):
            if sel is None:
                slots = st["idx"][start[b]:start[b + 1]].long()
            else:
                pick = sel[b, h][sel[b, h] >= 0].long()
                j = (pick[:, None] * case["page"] + torch.arange(case["page"], device=DEV)).flatten()
                j = j[j < t]
                slots = st["ids"][start[b] + j // case["page"]].long() * case["page"] + j % case["page"]
            rows = slice(h * group, (h + 1) * group)
            o[b, rows], lse[b, rows] = _exact_attend(
                st, st["q"][b, rows].double(), _exact_rows(st, "k", slots, h), _exact_rows(st, "v", slots, h))
    return (o, lse) if sel is None else (sel, o, lse)
