"""GPU tests of attention calls that have nothing to do (no sequence, or no
new token): they succeed, and the status of the workspace that they return is
good, whatever its memory held before."""
import pytest
import torch

from paged_kv_extend_gb300 import pkx

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
HQ, HKV, D = 8, 2, 128


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkx.load_library()


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _calls(b):
    """Each attention call of no sequence (b = 0), or of b sequences without
    new tokens (the extend forms alone)."""
    row = lambda h: torch.zeros(0, h, D, dtype=torch.bfloat16, device=DEV)
    pool = torch.zeros(16, HKV, D, dtype=torch.bfloat16, device=DEV)
    fp4 = (torch.zeros(16, HKV, D // 2, dtype=torch.uint8, device=DEV),
           torch.zeros(16, HKV, D // 16, dtype=torch.float8_e4m3fn, device=DEV)) * 2
    q, o, ke, ve = row(HQ), row(HQ), row(HKV), row(HKV)
    ptr, none = _i32(*([0] * (b + 1))), _i32()
    long = torch.zeros(0, dtype=torch.int64, device=DEV)
    calls = dict(
        extend=lambda: pkx.extend_attention_fwd(q, ke, ve, o, pool, pool, ptr, ptr, none),
        ragged_paged=lambda: pkx.extend_attention_fwd_ragged_paged(q, ke, ve, o, pool, pool, ptr, ptr, none),
        unified=lambda: pkx.extend_attention_fwd_unified(q, o, pool, pool, ptr, ptr, long, _i32(*([0] * b))),
        extend_fp4=lambda: pkx.extend_attention_fwd_fp4(q, ke, ve, o, *fp4, ptr, ptr, none),
        streaming=lambda: pkx.extend_attention_fwd_streaming(q, ke, ve, o, pool, pool, ptr, ptr, none, 64, 4))
    if b == 0:
        calls.update(
            decode=lambda: pkx.decode_attention_fwd(q, o, pool, pool, ptr, none),
            decode_fp4=lambda: pkx.decode_attention_fwd_fp4(q, o, *fp4, ptr, none),
            decode_streaming=lambda: pkx.decode_attention_fwd_streaming(q, o, pool, pool, ptr, none, 64, 4))
    return calls


@pytest.mark.parametrize("b", [0, 3])
def test_status_of_an_empty_call(b):
    for name, call in _calls(b).items():
        size = call().numel()
        torch.cuda.synchronize()
        torch.full((size,), 5, dtype=torch.uint8, device=DEV)  # memory that the next workspace gets
        ws = call()
        assert pkx.workspace_status(ws) == 0, name


def test_a_given_workspace_is_left_alone():
    ws = torch.full((1 << 20,), 7, dtype=torch.uint8, device=DEV)
    q = torch.zeros(0, HQ, D, dtype=torch.bfloat16, device=DEV)
    pool = torch.zeros(16, HKV, D, dtype=torch.bfloat16, device=DEV)
    got = pkx.decode_attention_fwd_streaming(q, q, pool, pool, _i32(0), _i32(), 64, 4, workspace=ws)
    assert got is ws and (ws == 7).all()
