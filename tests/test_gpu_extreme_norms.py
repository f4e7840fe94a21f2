"""GPU tests of the query / key norm over bf16's whole range: rows whose squares
fp32 does not hold."""
import pytest
import torch

import step_reference as R
from paged_kv_extend_gb300 import pkx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _check(out, ref, size):
    """One rounding to bf16 (2^-8 of the value; below 2^-126 half a step is 2^-134)
    and fp32 work: the sum of at most 256 squares (2^-16, halved by the root),
    rsqrt, products: 2^-16 of the elements that enter.  A product below 2^-126
    keeps 2^-149 of each of its factors' two terms, far below 2^-134."""
    out = out.double().cpu()
    nan = ref.isnan()
    assert torch.equal(out.isnan(), nan)
    err = (out - ref).abs() - 2.0 ** -8 * ref.abs() - 2.0 ** -16 * size - 2.0 ** -133
    assert not (err[~nan] > 0).any()


SCALES = [2.0 ** e for e in (-130, -126, -110, -75, -62, -50, -49, 0, 50, 58, 59, 60, 63, 64, 100, 124)]


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -140, 2.0 ** -101, 2.0 ** -99, 1e-6, 2.0 ** 100])
@pytest.mark.parametrize("d,r,leaved,hq", [(128, 128, False, 8), (64, 32, True, 3), (256, 256, False, 2), (40, 16, True, 5)])
def test_rows_of_every_size(d, r, leaved, hq, eps):
    """Rows of one size each, and rows whose elements differ by up to 2^30; heads of
    ordinary size among them keep theirs."""
    g = torch.Generator().manual_seed(d + hq)
    n = 2 * len(SCALES) + 1
    x = torch.randn(n, hq, d, generator=g).clamp(-4, 4)
    for i, f in enumerate(SCALES):
        x[i] *= f
        x[len(SCALES) + i] *= f * 2.0 ** torch.randint(-30, 1, (hq, d), generator=g)
    x[:, hq // 2] = torch.randn(n, d, generator=g)
    x[-1] = 0.0
    x[-1, 0, 3] = 3.3e38
    q = x.bfloat16()
    assert q.isfinite().all()
    w = (1 + torch.randn(d, generator=g) * 0.3).bfloat16()
    w[5] = 60.0
    angle = torch.rand(9, r // 2, generator=g, dtype=torch.float64) * 6.3
    table = torch.cat([angle.cos(), angle.sin()], 1).float()
    pos = torch.randint(0, 9, (n,), generator=g)
    on = [t.to(DEV) for t in (q, pos, table, w)]
    qo, ko = pkx.qk_norm_rope(on[0], on[0], on[1], on[2], q_weight=on[3], k_weight=on[3], eps=eps, interleaved=leaved)
    ref, size = R.rope(q, w, torch.tensor(eps).double(), 0.0, pos, table, leaved, None)
    big = ref.abs() > 3.38e38  # nothing of the kind
    assert not big.any()
    _check(qo, ref, size)
    assert torch.equal(qo.nan_to_num(7.0), ko.nan_to_num(7.0))


def test_infinite_rows():
    """inf / sqrt(inf): NaN where the infinity stood, 0 elsewhere; NaN rows are NaN."""
    q = torch.randn(5, 3, 128).bfloat16()
    q[1, 1, 7], q[2, 0, 0], q[3, 2, 9], q[4, 1, 5] = float("inf"), float("-inf"), float("nan"), 3.3e38
    q[4, 1, 6] = float("inf")
    w = torch.ones(128, dtype=torch.bfloat16)
    ref, size = R.rope(q, w, 1e-6, 0.0, None, None, False, None)
    out, _ = pkx.qk_norm_rope(q.to(DEV), q.to(DEV), q_weight=w.to(DEV))
    _check(out, ref, size)
    assert out[1, 1, 7].isnan() and not out[1, 1, :7].any() and not out[4, 1, 5].any()
