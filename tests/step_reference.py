"""64-bit reference of a decode step's operators: norm and rotation, page bounds
and selection, attention over a list of slots.  CPU tensors, plain loops."""
import torch

FP8_MAX = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}


def rope(x, weight, eps, offset, positions, cos_sin, interleaved, pair_axis):
    """(float64 rows, magnitude of the products that make each element)."""
    y = x.double()
    if weight is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * (weight.double() + offset)
    out, size = y.clone(), y.abs()
    if cos_sin is None:
        return out, size
    r = cos_sin.shape[1]
    pos = positions if positions.dim() == 2 else positions[None]
    for i in range(r // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        axis = 0 if pair_axis is None else int(pair_axis[i])
        ok = torch.zeros(x.shape[0], dtype=torch.bool)
        p = torch.zeros(x.shape[0], dtype=torch.int64)
        if axis < pos.shape[0]:
            p = pos[axis]
            ok = (p >= 0) & (p < cos_sin.shape[0])
            p = torch.where(ok, p, 0)
        c, s = (torch.where(ok, cos_sin[p, j].double(), float("nan"))[:, None] for j in (i, r // 2 + i))
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        size[..., a] = size[..., b] = y[..., a].abs() + y[..., b].abs()
    return out, size


def bounds(k, ids, lens, page, into):
    out = into.clone()
    for p, t in zip(ids.tolist(), lens.tolist()):
        if 0 <= p < into.shape[0] and t > 0:
            rows = k[p * page:p * page + min(t, page)].to(into.dtype)
            out[p, :, 0], out[p, :, 1] = rows.amin(0), rows.amax(0)
    return out


def _tree32(t):
    while t.shape[-1] > 1:
        t = (t[..., 0::2] + t[..., 1::2]).float().double()
    return t[..., 0]


def scores(q, box):
    """fp32 scores [pages] of one KV head: q [group, d], box [pages, 2, d]."""
    pos = torch.zeros(q.shape[1], dtype=torch.float64)
    neg = pos.clone()
    for x in q.double():
        pos = (pos + torch.where(x > 0, x, 0.0)).float().double()
        neg = (neg + torch.where(x < 0, x, 0.0)).float().double()
    lo = _tree32((box[:, 0].double() * neg).float().double())
    hi = _tree32((box[:, 1].double() * pos).float().double())
    return (lo + hi).float()


def select(q, box, indptr, ids, top, first, last):
    b, hq, _ = q.shape
    hkv = box.shape[1]
    out = torch.full((b, hkv, top), -1, dtype=torch.int32)
    for i in range(b):
        pages = ids[int(indptr[i]):int(indptr[i + 1])].long()
        n = len(pages)
        for h in range(hkv):
            if n <= top:
                out[i, h, :n] = torch.arange(n)
                continue
            s = scores(q[i].unflatten(0, (hkv, -1))[h], box[pages, h]).tolist()
            rank = sorted(range(first, n - last), key=lambda p: (0 if s[p] != s[p] else 1, -s[p] if s[p] == s[p] else 0, p))
            out[i, h] = torch.tensor(sorted([*range(first), *range(n - last, n), *rank[:top - first - last]]))
    return out


def attend(q, k, v, scale, cap=0.0):
    """One KV head: q [g, d], k / v [t, d] float64 -> (o, lse, sum p |v|)."""
    if not k.shape[0]:
        return torch.zeros_like(q), torch.full((q.shape[0],), float("-inf"), dtype=q.dtype), torch.zeros_like(q)
    s = (q @ k.T) * scale
    if cap > 0:
        s = cap * torch.tanh(s / cap)
    p = torch.softmax(s, -1)
    return p @ v, torch.logsumexp(s, -1), p @ v.abs()


def check_attention(o, lse, ref, cap=0.0):
    """o bf16 and lse against the reference's (o, lse, sum p |v|).  P and o are
    each rounded to bf16 (2^-8 of the value); the fp32 sums, exp2 and the merge
    stay below 2^-11 of sum p |v|; a capped logit is off by cap * 2^-10 (the
    hardware tanh), which moves p by twice that."""
    ro, rl, size = ref
    o, lse = o.double().cpu(), lse.double().cpu()
    bound = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -11 + 2 * cap * 2.0 ** -10) * size + 1e-30
    bad = (o - ro).abs() > bound
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs off by up to {((o - ro).abs() / bound).max()} bounds"
    empty = rl == float("-inf")
    assert torch.equal(lse == float("-inf"), empty)
    assert (lse - rl)[~empty].abs().max().item() <= 1e-3 + cap * 2.0 ** -10 if (~empty).any() else True
