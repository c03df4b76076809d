"""PagedStack.read into caches of other strides, on the host (stand-ins as in
test_kv8_stack_host.py): over 8-bit pages a pair of differing strides is refused before any
layer is read; strides that mean nothing do not matter."""
import pytest

torch = pytest.importorskip("torch")
import decode_qwen2_block_gb300 as blk  # noqa: E402
from test_kv8_stack_host import made  # noqa: E402,F401


def cache(slots, D=64, last=1):
    return torch.zeros((2, slots, D * last), dtype=torch.float16)[..., ::last]


def test_a_pair_of_differing_strides_is_refused_before_anything_is_read(made):  # noqa: F811
    make, calls, _ = made
    pg = make(kv8=True)
    pg.step(torch.zeros(5, 8), [5])
    del calls[:]
    ok = (cache(9), cache(9))
    for bad in ((cache(9), cache(12)), (cache(9), cache(9).transpose(0, 1).contiguous().transpose(0, 1)),
                (cache(9, last=2), cache(9, last=2)), (cache(9), cache(9, last=2))):
        for caches in ([ok, bad], [bad, ok]):
            with pytest.raises(blk.BlkError) as e:
                pg.read(0, caches=caches)
            assert e.value.status == blk.BLK_ERR_SHAPE
    assert not calls
    same = [(cache(12), cache(12)), (cache(9)[:, :7], cache(9)[:, 2:])]
    assert pg.read(0, caches=same) == same and [c[0] for c in calls] == ["read"] * 2


def test_over_fp16_pages_any_strides_are_served(made):  # noqa: F811
    make, calls, _ = made
    pg = make()
    pg.step(torch.zeros(5, 8), [5])
    for p in pg.pools:
        for t in p:
            t.normal_()
    caches = [(cache(9), cache(12)), (cache(9, last=2), cache(9).transpose(0, 1).contiguous().transpose(0, 1))]
    pg.read(0, caches=caches)
    for pool, pair in zip(pg.pools, caches):
        for p, t in zip(pool, pair):
            assert torch.equal(t[:, :5], p[int(pg.table[0, 0]), :, :5]) and (t[:, 5:] == 0).all()


def test_strides_that_mean_nothing(made):  # noqa: F811
    make, calls, _ = made
    pg = make(kv8=True)
    pg.step(torch.zeros(1, 8), [1])                      # one slot: its stride is never taken
    k, v = cache(9), cache(9)
    caches = [(k, v.as_strided((2, 9, 64), (9 * 64, 32, 1)))] * 2
    assert pg.read(0, caches=caches) == caches
