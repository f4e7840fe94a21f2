"""CPU tests of the sizes at which a decode step's operators stop, and of what the
binding does with numbers and shapes that do not fit (nothing reaches a GPU)."""
import pytest
import torch

from paged_kv_extend_gb300 import build as pkx_build
from paged_kv_extend_gb300 import pkx

P = 0x10000  # an aligned address that no check dereferences


@pytest.fixture(scope="module")
def lib():
    pkx_build.build()
    return pkx.load_library()


@pytest.mark.parametrize("hq,hkv,batch,page,top", [
    (8, 1, 1, 2 ** 31 - 2, 1), (32, 1, 1, 2 ** 31 - 2, 1), (8, 1, 1, 2 ** 31 - 1024, 1),
    (34, 1, 1, 2 ** 31 - 64, 1), (8, 2, 4, 2 ** 26 - 64, 4), (8, 1, 1, 2 ** 20 - 1, 2048),
])
def test_lists_of_selected_pages_end_below_the_int_range(lib, hq, hkv, batch, page, top):
    """Runs, tiles and blocks of slots reach past the end of a list of keys by up to
    some hundred; their numbers have to stay 32-bit."""
    assert lib.pkx_decode_attention_fwd_pages(
        P, P, P, P, P, P, 40, P, page, P, top, batch, hq, hkv, 64, 64, 64, 64, 64, 64, 640, 0.0, 0.0, 0, 1.0, 1.0,
        None, P, 1 << 60, None) == pkx.PKX_EUNSUPPORTED
    if batch == 1:
        assert pkx.decode_pages_workspace_size(batch, hq, hkv, 64, 64, page, top) == 0


@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 1024, 2 ** 40])
@pytest.mark.parametrize("hq", [8, 34])
def test_lists_of_shared_prefixes_end_below_the_int_range(lib, n, hq):
    assert lib.pkx_decode_attention_fwd_shared(
        P, P, P, P, P, P, n, P, P, 1, 2, hq, 1, 64, 64, 64, 64, 64, 64, 640, 0.0, 0.0, 0, 1.0, 1.0, None, P, 1 << 60,
        None) == pkx.PKX_EUNSUPPORTED


def test_pages_of_bounds_end_below_the_int_range(lib):
    bounds = lambda page: lib.pkx_update_page_bounds(P, 64, 64, 0, page, 1, 1, 64, P, None, 1, P, None)
    assert bounds(2 ** 30 + 1) == pkx.PKX_EUNSUPPORTED and bounds(2 ** 31 - 1) == pkx.PKX_EUNSUPPORTED


@pytest.mark.parametrize("shape", [(6, 64), (64,), (), (3, 2, 32), (3, 2, 64, 1)])
def test_rows_of_another_shape_are_refused(shape):
    with pytest.raises(ValueError, match="v must be a CUDA bf16 tensor"):
        pkx._rows_at(torch.zeros(shape, dtype=torch.bfloat16), (3, 2, 64), -1, "v")
    assert pkx._rows_at(x := torch.zeros(3, 2, 64, dtype=torch.bfloat16), (3, 2, 64), -1, "v") == (x.data_ptr(), 128, 64)


def test_workspace_sizes_past_the_c_int_range():
    assert pkx.decode_pages_workspace_size(2, 8, 2, 64, 64, 16, 4) > 0
    assert pkx.decode_pages_workspace_size(2, 8, 2, 64, 64, 2 ** 32 + 16, 4) == 0
    assert pkx.decode_pages_workspace_size(2, 8, 2, 64, 64, 16, 2 ** 32 + 4) == 0
