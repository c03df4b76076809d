"""GPU tests of where a read of an 8-bit cache may write: K's and V's rows in one buffer, and
the refusal of rows over each other."""
import pytest
import torch

import decode_qwen2_block_gb300 as blk
from kv8_reference import quantise, same, values
from test_kv8_gpu import MARK, block, pools

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,kv,dim", [(1, 1, 64), (37, 2, 64), (37, 4, 128), (5, 1, 128)])
def test_rows_of_k_and_v_in_one_buffer(n, kv, dim):
    b = block(kv * 2, kv, dim)
    x = torch.randn((n, kv, dim), device="cuda").half()
    y = torch.randn((n, kv, dim), device="cuda").half()
    p = pools(-(-n // 16), kv, 16, dim)
    slots = torch.arange(n, device="cuda")
    b.page_append_kv8(x, y, slots, *p)
    want = [values(*quantise(t)) for t in (x, y)]
    for shape, pick in (((n, 2, kv, dim), lambda t, i: t[:, i]), ((2, n, kv, dim), lambda t, i: t[i]),
                        ((n, kv, 2, dim), lambda t, i: t[:, :, i]),
                        ((kv, n, 2, dim), lambda t, i: t[:, :, i].transpose(0, 1)),
                        ((kv, 2, n, dim), lambda t, i: t[:, i].transpose(0, 1))):
        for turn in (0, 1):
            both = torch.full(shape, MARK, dtype=torch.float16, device="cuda")
            b.page_read_kv8(slots, *p, pick(both, turn), pick(both, 1 - turn))
            b.check()
            assert same(pick(both, turn), want[0]) and same(pick(both, 1 - turn), want[1]), shape


@pytest.mark.parametrize("n,kv,dim", [(1, 1, 64), (37, 2, 64), (37, 4, 128), (5, 1, 128)])
def test_rows_over_each_other_are_refused(n, kv, dim):
    b = block(kv * 2, kv, dim)
    p = pools(-(-n // 16), kv, 16, dim)
    slots = torch.arange(n, device="cuda")
    buf = torch.full((3 * n * kv * dim,), MARK, dtype=torch.float16, device="cuda")
    size = n * kv * dim

    def rows(at, head_major=False):
        t = buf[at:at + size]
        return t.view(kv, n, dim).transpose(0, 1) if head_major else t.view(n, kv, dim)

    for major in (False, True):
        for at in (0, 8, dim - 8, size - 8, size - dim):
            for k, v in ((rows(0, major), rows(at, major)), (rows(at, major), rows(0, major))):
                with pytest.raises(blk.BlkError) as e:
                    b.page_read_kv8(slots, *p, k, v)
                assert e.value.status == blk.BLK_ERR_SHAPE
    torch.cuda.synchronize()
    assert (buf == MARK).all()
