"""A plain float64 implementation of the 4-bit pool and of attention with a
window and first tokens that stay visible, for the tests.  Written from the
definitions: nearest values are found by search over the value tables, and
attention is a loop over sequences and heads."""
import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the 127 non-negative finite e4m3 values, code order
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
                 for e in range(16) for m in range(8)][:127])


def nearest(table, x):
    """Index of the table value nearest to x >= 0; ties to the even index,
    past the last value the last one."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = x - table[lo], table[hi] - x
    pick_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    return np.where(x >= table[-1], len(table) - 1, np.where(pick_lo, lo, hi))


def pack(x, scale):
    """bf16 rows [n, h, d] -> (codes uint8 [n, h, d / 2], block scales uint8)."""
    f = x.float().numpy()
    with np.errstate(all="ignore"):
        q = (f / np.float32(scale)).astype(np.float32).reshape(*f.shape[:2], -1, 16)
        nan = np.isnan(q).any(-1)
        amax = np.nanmax(np.where(np.isnan(q), 0, np.abs(q)), axis=-1)
        sc = nearest(E4M3, (amax / np.float32(6)).astype(np.float32))
        s = E4M3[sc][..., None]
        ratio = np.abs(q).astype(np.float64) / np.where(s > 0, s, 1.0)
        mag = nearest(E2M1, np.where(np.isnan(ratio), 0, ratio))
        code = mag | np.where(np.signbit(q), 8, 0)
        code = np.where((s > 0) & ~nan[..., None], code, 0).astype(np.uint8)
    sc = np.where(nan, 0x7F, sc).astype(np.uint8)
    code = code.reshape(*f.shape[:2], -1, 2)
    return (torch.from_numpy(code[..., 0] | (code[..., 1] << 4)), torch.from_numpy(sc))


def unpack(codes, bscale, scale=1.0):
    """float64 values of packed rows (bscale as uint8 or float8_e4m3fn)."""
    c = codes.cpu().numpy()
    b = bscale.cpu().view(torch.uint8).numpy()
    nib = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], 2 * c.shape[-1])
    val = E2M1[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    table = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])
    return torch.from_numpy(val * np.repeat(table[b], 16, axis=-1)) * float(np.float32(scale))


def visible(qpos, n_keys, window, first):
    """[len(qpos), n_keys] truth values."""
    j = torch.arange(n_keys)[None]
    back = qpos[:, None] - j
    ok = back >= 0
    if window > 0:
        ok &= (back <= window) | (j < first)
    return ok


def attend(q, k, v, ok, scale, cap=0.0, sinks=None):
    """q [n, hq, d], k / v [t, hkv, d] float64, ok [n, t].  Returns o, lse,
    sum_j p_j |v_j| and the largest sum_i |q_i k_i| of each (row, head)."""
    n, hq, d = q.shape
    group = hq // k.shape[1]
    o = torch.zeros(n, hq, v.shape[2], dtype=torch.float64)
    lse = torch.full((n, hq), float("-inf"), dtype=torch.float64)
    av, aq = torch.zeros_like(o), torch.zeros(n, hq, dtype=torch.float64)
    if sinks is not None:
        lse[:] = sinks.double()
    if not k.shape[0]:
        return o, lse, av, aq
    for h in range(hq):
        kk, vv = k[:, h // group], v[:, h // group]
        s = (q[:, h] @ kk.T) * scale
        if cap > 0:
            s = cap * torch.tanh(s / cap)
        s = s.masked_fill(~ok, float("-inf"))
        if sinks is not None:
            s = torch.cat([s, sinks[h].double().expand(n, 1)], 1)
        lse[:, h] = torch.logsumexp(s, -1)
        p = torch.exp(s - torch.where(torch.isinf(lse[:, h]), 0.0, lse[:, h])[:, None])
        p = p[:, :kk.shape[0]]
        o[:, h], av[:, h] = p @ vv, p @ vv.abs()
        aq[:, h] = (q[:, h].abs() @ kk.abs().T).masked_fill(~ok, 0.0).amax(-1)
    return o, lse, av, aq


def check(o, lse, ref, d, scale, p_step, what="", tanh_step=0.0):
    """o (bf16) and lse (fp32) against attend()'s result.

    Logits: d fp32 products summed with at most one rounding (or truncation,
    2^-23) a step, so |ds| <= d 2^-23 sum|q k| scale, and a few more ulp of the
    logit and of the exponent (2^-20 of sum|q k| scale, 2^-18 absolute).  P is
    rounded to a type of half step p_step and o to bf16 (2^-8): |do| <= 2^-8
    |o| + (p_step + 2 |ds|) sum p |v|.  lse errs by |ds| (and 2^-22 |lse|).
    tanh_step: relative error of the tanh behind a logit cap (2^-11 for
    tanh.approx), of a logit of at most sum |q k| scale."""
    ro, rl, av, aq = ref
    o, lse = o.detach().cpu().double(), lse.detach().cpu().double()
    ds = (d * 2.0 ** -23 + 2.0 ** -20 + tanh_step) * aq * scale + 2.0 ** -18
    assert torch.equal(torch.isinf(lse), torch.isinf(rl)), f"{what}: lse finiteness"
    fin = torch.isfinite(rl)
    err = (lse - rl)[fin].abs() - (ds + 2.0 ** -22 * rl.abs())[fin]
    assert not err.numel() or err.max() <= 0, f"{what}: lse off by {err.max().item():.2e} too much"
    tol = 2.0 ** -8 * ro.abs() + (p_step + 2 * ds)[..., None] * av + 1e-30
    assert torch.isfinite(o).all(), f"{what}: non-finite output"
    over = (o - ro).abs() - tol
    assert over.max() <= 0, f"{what}: o off by {over.max().item():.2e} too much"


def extend(wl, k_prefix, v_prefix, k_ext, v_ext, window=-1, first=0, cap=0.0, sinks=None, masks=None):
    """attend() over every sequence of a drawn workload: its prefix rows
    (float64 [P, hkv, d] each) and its extend rows."""
    out, q0, p0 = [], 0, 0
    for b, (p, e) in enumerate(zip(wl.prefix_lens, wl.extend_lens)):
        k = torch.cat([k_prefix[p0:p0 + p], k_ext[q0:q0 + e].double()])
        v = torch.cat([v_prefix[p0:p0 + p], v_ext[q0:q0 + e].double()])
        pos = torch.arange(e) + p
        ok = visible(pos, p + e, window, first)
        if masks is not None:
            ok = masks[b].bool()
            if window > 0:
                ok = ok & (pos[:, None] - torch.arange(p + e)[None] <= window)
        out.append(attend(wl.q[q0:q0 + e].double(), k, v, ok, wl.sm_scale, cap, sinks))
        q0, p0 = q0 + e, p0 + p
    return [torch.cat(x) for x in zip(*out)]
