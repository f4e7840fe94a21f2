"""GPU test of the quantising write over all pairs of a block's largest
element and another one: every mantissa of both, every distance of exponents
at which the other one does not surely round to zero, and block scales of
every kind (subnormal, normal, saturating, zero), bit for bit against the
plain implementation in fp4_reference.py."""
import math

import pytest
import torch

import fp4_reference as R
from paged_kv_extend_gb300 import pkx

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkx.load_library()


def _blocks(top, others):
    """Blocks of 16 for each value of top [m]: the value, then 15 of others
    [m, n], until all are used.  Signs alternate, and change from block to block."""
    m, n = others.shape
    pad = -n % 15
    others = torch.cat([others, others[:, :pad]], 1).view(m, -1, 15)
    x = torch.cat([top[:, None, None].expand(m, others.shape[1], 1), others], 2).reshape(-1, 16)
    sign = (torch.arange(x.numel()).view_as(x) + torch.arange(x.shape[0])[:, None]) % 2
    return torch.where(sign == 0, x, -x).bfloat16()[:, None]


def _check(x, scale):
    c, b = R.pack(x, scale)
    n = x.shape[0]
    kc = torch.full((n, 1, 8), 0xAA, dtype=torch.uint8, device=DEV)
    kb = torch.full((n, 1, 1), 0x55, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    pkx.set_kv_buffer_fp4(kc, kb, None, None, torch.arange(n, device=DEV), x.to(DEV), k_scale=scale)
    assert torch.equal(kb.view(torch.uint8).cpu(), b)
    assert torch.equal(kc.cpu(), c)
    return b


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -7, 2.0 ** 64, 2.0 ** -64, 0.3, 1.7e-3, 2.0 ** 65, 1.9999999])
def test_every_pair_of_mantissas(scale):
    mant = 1 + torch.arange(128).double() / 128
    # an element below a sixteenth of a quarter of a sixth of the largest rounds
    # to zero: with distances up to 7 the codes 0 to 7 are all met from both sides
    dist = (mant[None, :] * 2.0 ** -torch.arange(8).double()[:, None]).flatten()
    seen = set()
    for e in (-11, -9, -8, -7, -6, -5, -4, -3, -2, 0, 7, 9, 10, 11, 12, 40):
        exp = e + math.floor(math.log2(scale))
        if not -118 <= exp <= 127:
            continue
        top = mant * 2.0 ** exp
        others = torch.minimum(dist[None, :] * 2.0 ** exp, top[:, None])
        x = _blocks(top, others)
        assert torch.isfinite(x.float()).all()
        seen |= set(_check(x, scale).flatten().tolist())
    # no scale, subnormal ones, the largest (the next code is NaN's)
    assert {0, 1, 2, 7, 8, 0x7E} <= seen and 0x7F not in seen


@pytest.mark.parametrize("scale", [2.0 ** -125, 3e-38, 1.0])
def test_every_pair_of_subnormals(scale):
    sub = torch.arange(1, 128).double() * 2.0 ** -133
    top = torch.cat([sub, torch.arange(128, 256).double() * 2.0 ** -133])
    others = torch.minimum(top[None, :], top[:, None])
    _check(_blocks(top, others), scale)
