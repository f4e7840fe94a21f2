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


@pytest.mark.parametrize("over", [dict(top_k=2 ** 32 + 4), dict(top_k=-2 ** 32 + 4), dict(first_pages=2 ** 32),
                                  dict(last_pages=2 ** 32 + 1), dict(first_pages=-2 ** 32), dict(top_k=4097)], ids=str)
def test_page_numbers_past_the_c_int_range(over):
    """They are refused, not cut to their low 32 bits."""
    q, box, i32 = _z(2, 4, 64), _z(30, 2, 2, 64), torch.int32
    ptr, ids = torch.tensor([0, 20, 30], dtype=i32, device=DEV), torch.arange(30, dtype=i32, device=DEV)
    a = dict(top_k=4, first_pages=1, last_pages=1)
    pkx.select_pages(q, box, ptr, ids, **a)
    with pytest.raises(pkx.PkxError):
        pkx.select_pages(q, box, ptr, ids, **{**a, **over})


def test_page_sizes_past_the_c_int_range():
    q, pool, i32 = _z(2, 4, 64), _z(64, 2, 64), torch.int32
    ptr, ids = torch.tensor([0, 2, 4], dtype=i32, device=DEV), torch.arange(4, dtype=i32, device=DEV)
    last, sel = torch.ones(2, dtype=i32, device=DEV), _z(2, 2, 2, dtype=i32)
    run = lambda page, ws=None: pkx.decode_attention_fwd_pages(q, torch.empty_like(q), pool, pool, ptr, ids, last, page, sel,
                                                               workspace=ws)
    ws = run(16)
    for page in (2 ** 32 + 16, -2 ** 32 + 16):
        with pytest.raises(pkx.PkxError):
            run(page)
        with pytest.raises(pkx.PkxError):
            run(page, ws)
        with pytest.raises(ValueError):
            pkx.update_page_bounds(pool, _z(4, 2, 2, 64), ids, page)
