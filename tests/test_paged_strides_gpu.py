"""GPU tests of tensors whose strides of a dimension of size one mean nothing: the smallest
batch as other code lays it out."""
import pytest
import torch

import decode_qwen2_block_gb300 as blk
from paged_reference import Batch
from test_paged_gpu import MARK, block, check_rows

pytestmark = pytest.mark.gpu


def _call(x, q, out):
    b = block(x.heads, x.kv, x.dim)
    ws = torch.empty(b.attn_paged_workspace_bytes(x.rows, len(x.hist)), dtype=torch.uint8,
                     device="cuda")
    b.attn_paged(x.descriptor(b), q, x.k_pages, x.v_pages, out, ws)
    b.check()


@pytest.mark.parametrize("heads,kv,dim", [(12, 2, 128), (4, 2, 64)])
def test_one_row_out_of_head_major_tensors(heads, kv, dim):
    x = Batch(heads, kv, dim, 64, [300], [1], seed=51)
    q = torch.empty((heads, 1, dim), dtype=torch.float16, device="cuda").transpose(0, 1)
    q.copy_(x.q)
    out = torch.full((heads, 1, dim), MARK, dtype=torch.float16, device="cuda").transpose(0, 1)
    assert q.stride(0) == out.stride(0) == dim
    _call(x, q, out)
    check_rows(x, out)


@pytest.mark.parametrize("rows,stride", [(3, 64), (1, 64), (3, 4096), (1, 8)])
def test_one_head_whatever_its_stride(rows, stride):
    x = Batch(1, 1, 64, 16, [70], [rows], seed=52)
    q = torch.empty((rows, 8192), dtype=torch.float16, device="cuda")[:, :64].unsqueeze(1)
    q.copy_(x.q)
    q = q.as_strided((rows, 1, 64), (q.stride(0), stride, 1))
    out = torch.full((rows, 1, 64), MARK, dtype=torch.float16, device="cuda")
    _call(x, q, out.as_strided((rows, 1, 64), (64, stride, 1)))
    check_rows(x, out)


@pytest.mark.parametrize("n,kv", [(1, 2), (5, 1), (1, 1)])
def test_append_takes_rows_of_differing_strides_where_they_mean_nothing(n, kv):
    """A row of a packed projection beside a contiguous one; one head of another stride."""
    dim = 64
    k = torch.randn((n, kv, dim), device="cuda").half()
    packed = torch.randn((n, 6, kv, dim), device="cuda").half()
    v = packed[:, 3] if n == 1 else packed[:, 0].contiguous()
    k = k.as_strided((n, kv, dim), (k.stride(0) if n > 1 else 3, 5 if kv == 1 else dim, 1))
    pools = [torch.full((3, kv, 16, dim), MARK, dtype=torch.float16, device="cuda") for _ in range(2)]
    slots = torch.tensor([40, 3, 17, -1, 0][:n], device="cuda")
    b = block(kv * 2, kv, dim)
    b.page_append(k, v, slots, *pools)
    b.check()
    for pool, rows in zip(pools, (k, v)):
        want = torch.full((48, kv, dim), MARK, dtype=torch.float16, device="cuda")
        want[slots[slots >= 0]] = rows[slots >= 0]
        assert torch.equal(pool.transpose(1, 2).reshape(48, kv, dim), want)


def test_strides_that_mean_something_are_still_refused():
    b = block(4, 2, 64)
    x = Batch(4, 2, 64, 16, [70], [2], seed=53)
    ws = torch.empty(b.attn_paged_workspace_bytes(2, 1), dtype=torch.uint8, device="cuda")
    out = torch.empty((2, 4, 64), dtype=torch.float16, device="cuda")
    for q, o in ((x.q.transpose(0, 1).contiguous().transpose(0, 1), out),
                 (x.q, torch.empty((4, 2, 64), dtype=torch.float16, device="cuda").transpose(0, 1)),
                 (x.q[:1].expand(2, 4, 64), out)):
        with pytest.raises(blk.BlkError) as e:
            b.attn_paged(x.descriptor(b), q, x.k_pages, x.v_pages, o, ws)
        assert e.value.status == blk.BLK_ERR_SHAPE
    k = torch.zeros((2, 2, 64), dtype=torch.float16, device="cuda")
    wide = torch.zeros((2, 3, 64), dtype=torch.float16, device="cuda")[:, :2]
    pools = [torch.zeros((3, 2, 16, 64), dtype=torch.float16, device="cuda") for _ in range(2)]
    with pytest.raises(blk.BlkError) as e:
        b.page_append(k, wide, torch.tensor([0, 1], device="cuda"), *pools)
    assert e.value.status == blk.BLK_ERR_SHAPE
