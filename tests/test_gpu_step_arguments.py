"""GPU tests of what the binding of a decode step's operators refuses."""
import pytest
import torch

from paged_kv_extend_gb300 import pkx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype, device=DEV)


def test_tensors_of_other_ranks():
    q, k, loc, i32 = _z(3, 4, 64), _z(3, 2, 64), _z(3, dtype=torch.int64), torch.int32
    pool, ptr, idx = _z(16, 2, 64), _z(4, dtype=i32), _z(1, dtype=i32)
    pages = lambda sel: pkx.decode_attention_fwd_pages(q, q.clone(), pool, pool, ptr, idx, ptr[:3], 8, sel)
    for call in (lambda: pkx.qk_norm_rope(q, k, q_out=_z(12, 64)), lambda: pkx.qk_norm_rope(q, k, k_out=_z(384)),
                 lambda: pkx.qk_norm_rope(q, k, cache_loc=loc, v=_z(6, 64), k_buffer=pool, v_buffer=pool.clone()),
                 lambda: pkx.update_page_bounds(pool, _z(()), idx, 8),
                 lambda: pkx.update_page_bounds(pool, _z(2, 256), idx, 8),
                 lambda: pages(_z((), dtype=i32)), lambda: pages(_z(6, 2, dtype=i32))):
        with pytest.raises(ValueError):
            call()
