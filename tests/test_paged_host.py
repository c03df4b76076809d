"""Host-side checks of the paged entry points that need no GPU."""
import ctypes

import pytest

import decode_qwen2_block_gb300 as blk
from decode_qwen2_block_gb300 import build as gpu_build


@pytest.fixture(scope="module")
def lib():
    gpu_build.build()
    return blk.load()


def test_null_handles_are_refused(lib):
    w, b = blk.BlkWeights(), blk.BlkPagedBatch()
    N = blk.BLK_ERR_NULL
    assert blk.blk_page_plan(None, 16, 1, 16, 16, 16, 1, 16, 1, 1, 16, 16, 16, 16, None) == N
    assert blk.blk_page_append(None, 16, 16, 64, 64, 16, 1, 16, 1, 16, 16, None) == N
    assert blk.blk_attn_paged(None, b, 16, 64, 16, 16, 16, 64, 16, 1 << 20, None) == N
    assert blk.blk_step_paged(None, w, b, 16, 16, 16, 16, 16, 16, 16, 1 << 20, None) == N
    one = (ctypes.c_void_p * 1)(16)
    assert blk.blk_step_paged_stack(None, (blk.BlkWeights * 1)(w), 1, b, one, one, 16, 16, 16, 16, 16,
                                    1 << 20, None) == N
    assert blk.blk_attn_paged_workspace_bytes(None, 1, 1, 1) == 0
    assert blk.blk_step_paged_workspace_bytes(None, 1, 1, 1) == 0


def test_the_page_status_has_a_text_of_its_own(lib):
    assert "paged" in blk.blk_status_str(blk.BLK_ERR_PAGE)


def test_the_batch_structure_is_laid_out_as_in_c():
    """blk_paged_batch: eleven 8-byte fields and page_size behind them."""
    assert blk.BlkPagedBatch.page_size.offset == 11 * 8
    assert ctypes.sizeof(blk.BlkPagedBatch) == 12 * 8
