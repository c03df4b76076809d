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


def test_the_tensor_calls_refuse_what_is_not_theirs(lib):
    """Tensors of another device, type or shape, and arguments that are no tensors, are
    refused before the library is called."""
    torch = pytest.importorskip("torch")
    from decode_qwen2_block_gb300 import _native
    args = (None, 0, 4, 2, 64)
    i64, f16 = torch.zeros(3, dtype=torch.int64), torch.zeros((3, 2, 64), dtype=torch.float16)
    pool = torch.zeros((5, 2, 16, 64), dtype=torch.float16)
    table = torch.zeros((3, 2), dtype=torch.int32)
    batch = blk.BlkPagedBatch()
    calls = [lambda: _native.page_plan(args, 16, i64, None, i64, table, i64, i64, i64, i64, None),
             lambda: _native.page_append(args, f16, f16, i64, pool, pool, None),
             lambda: _native.page_append(args, f16, f16, i64, f16, pool, None),
             lambda: _native.attn_paged(args, batch, f16, pool, pool, f16, i64, None)]
    for c in calls:
        with pytest.raises(blk.BlkError) as e:
            c()
        assert e.value.status == blk.BLK_ERR_SHAPE
    calls = [lambda: _native.page_plan(args, 16, i64), lambda: _native.page_append(args, 1, 2, 3, 4, 5, 6),
             lambda: _native.page_plan(args, "16", i64, None, i64, table, i64, i64, i64, i64, None),
             lambda: _native.page_plan(args[:4], 16, i64, None, i64, table, i64, i64, i64, i64, None),
             lambda: _native.attn_paged(args, i64, f16, pool, pool, f16, i64, None),
             lambda: _native.attn_paged(args, bytearray(8), f16, pool, pool, f16, i64, None)]
    for c in calls:
        with pytest.raises(TypeError):
            c()
