"""GPU tests of the 4-bit write and read back over more than 2^31 blocks or
chunks in one call: only the memory sets a limit."""
import pytest
import torch

import fp4_reference as R
from paged_kv_extend_gb300 import pkx

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
HKV, D = 8, 128


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    pkx.load_library()


def _rows(n, seed):
    return torch.randn(n, HKV, D, generator=torch.Generator().manual_seed(seed)).bfloat16()


def test_read_back():
    """2^31 + 2^20 chunks: 34 GB of bf16 rows.  The rows around the border and
    at the end are compared, and all of them on the device."""
    slots, n = 1009, (1 << 31) // (HKV * D // 8) + (1 << 13)
    c, b = R.pack(_rows(slots, 1), 0.5)
    kc, kb = c.to(DEV), b.view(torch.float8_e4m3fn).to(DEV)
    # slot i mod 1009, but the last row outside the pool
    idx = (torch.arange(n, device=DEV) % slots).to(torch.int32)
    idx[-1] = slots
    k, _ = pkx.get_kv_buffer_fp4(kc, kb, None, None, idx, 0.5)
    want = (R.unpack(c, b).float() * 0.5).bfloat16().to(DEV)
    border = (1 << 31) // (HKV * D // 8)
    for at in (0, border - 2, border, n - 5):
        assert torch.equal(k[at:at + 4], want[torch.arange(at, at + 4) % slots])
    assert not k[-1].any()
    whole = (n - 1) // slots * slots
    by_slot = k[:whole].view(-1, slots, HKV, D)
    for i in range(0, by_slot.shape[0], 2048):
        assert (by_slot[i:i + 2048] == want).all()


def test_write():
    """2^31 + 2^19 blocks: the tokens' rows are one row repeated (a token
    stride of 0) and most go to no slot."""
    n = (1 << 31) // (HKV * D // 16) + (1 << 13)
    x = _rows(1, 2)
    c, b = R.pack(x, 0.5)
    border = (1 << 31) // (HKV * D // 16)
    tokens = [0, 1, border - 1, border, border + 7, n - 1]
    loc = torch.full((n,), -1, dtype=torch.int64, device=DEV)
    loc[torch.tensor(tokens, device=DEV)] = torch.arange(len(tokens), device=DEV)
    kc = torch.full((len(tokens) + 1, HKV, D // 2), 0xAA, dtype=torch.uint8, device=DEV)
    kb = torch.full((len(tokens) + 1, HKV, D // 16), 0x55, dtype=torch.uint8, device=DEV)
    pkx.set_kv_buffer_fp4(kc, kb.view(torch.float8_e4m3fn), None, None, loc, x.to(DEV).expand(n, HKV, D),
                          k_scale=0.5)
    for got, want, before in ((kc, c, 0xAA), (kb, b, 0x55)):
        assert torch.equal(got[:-1].cpu(), want.expand(len(tokens), -1, -1))
        assert (got[-1] == before).all()
