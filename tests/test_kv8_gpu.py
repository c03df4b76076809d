"""GPU tests of the 8-bit paged cache's append and read: codes, scales and values bit for
bit against the definition in 64 bits (tests/kv8_reference.py)."""
import pytest
import torch

import decode_qwen2_block_gb300 as blk
from kv8_reference import BLOCK, E5M2, NAN_SCALE, quantise, same, values
from test_paged_gpu import MARK, block

pytestmark = pytest.mark.gpu
E5 = torch.float8_e5m2
FILL = 77                 # what codes and scales hold where nothing may be written


def pools(n_pages, kv, page, dim, fill=FILL):
    def make(last):
        return torch.full((n_pages, kv, page, last), fill, dtype=torch.uint8, device="cuda")
    return [make(dim), make(dim), make(dim // BLOCK).view(E5), make(dim // BLOCK).view(E5)]


def by_slot(pool):
    """[n_pages, kv, page, x] as bytes [slots, kv, x]."""
    return pool.view(torch.uint8).transpose(1, 2).reshape(-1, pool.shape[1], pool.shape[3])


def check_append(k, v, slots, p):
    keep = slots >= 0
    for rows, codes, scales in ((k, p[0], p[2]), (v, p[1], p[3])):
        c, s = quantise(rows)
        want_c, want_s = torch.full_like(by_slot(codes), FILL), torch.full_like(by_slot(scales), FILL)
        want_c[slots[keep]], want_s[slots[keep]] = c[keep], s[keep]
        got_c, got_s = by_slot(codes).clone(), by_slot(scales)
        assert torch.equal(got_s, want_s)
        nan = (want_s == NAN_SCALE).repeat_interleave(BLOCK, -1)     # those codes may be any
        got_c[nan] = want_c[nan] = 0
        assert torch.equal(got_c, want_c)


def rows_of(layout, n, kv, dim, gen):
    """k and v [n, kv, dim]: rows, slices of a fused projection's rows, slots of a contiguous
    cache; magnitudes from fp16's least to its greatest."""
    if layout == "rows":
        x = torch.randn((2, n, kv, dim), generator=gen, device="cuda").half()
        k, v = x[0], x[1]
    elif layout == "packed":
        x = torch.randn((n, 6 * kv * dim), generator=gen, device="cuda").half()
        k, v = (x[:, i * kv * dim:(i + 1) * kv * dim].unflatten(1, (kv, dim)) for i in (4, 5))
    else:
        x = torch.randn((2, kv, n + 9, dim), generator=gen, device="cuda").half()
        k, v = x[0, :, 4:4 + n].transpose(0, 1), x[1, :, 4:4 + n].transpose(0, 1)
    for t in (k, v):
        e = torch.randint(-26, 16, (n, kv, 1), generator=gen, device="cuda").double()
        t.copy_((t.double() * torch.where(e > 10, 0.2, 1.0) * 2.0 ** e).clamp(-65504, 65504).half())
    return k, v


@pytest.mark.parametrize("kv,dim,page", [(2, 128, 64), (8, 64, 16), (1, 128, 128), (1, 64, 32)])
@pytest.mark.parametrize("n", [1, 3, 77, 5000])
@pytest.mark.parametrize("layout", ["rows", "packed", "heads"])
def test_append_and_read(kv, dim, page, n, layout):
    gen = torch.Generator("cuda")
    gen.manual_seed(n)
    n_pages = -(-n // page) + 2
    k, v = rows_of(layout, n, kv, dim, gen)
    slots = torch.randperm(n_pages * page, generator=gen, device="cuda")[:n]
    if n > 3:
        slots[n // 2] = -1
    p = pools(n_pages, kv, page, dim)
    b = block(kv * 2, kv, dim)
    b.page_append_kv8(k, v, slots, *p)
    b.check()
    check_append(k, v, slots, p)
    back = [t.clone(memory_format=torch.preserve_format) for t in (k, v)]
    if layout == "packed":      # the same strides, the columns between them marked
        whole = torch.full((n, 6 * kv * dim), MARK, dtype=torch.float16, device="cuda")
        back = [whole[:, i * kv * dim:(i + 1) * kv * dim].unflatten(1, (kv, dim)) for i in (1, 3)]
    elif layout == "heads":
        whole = torch.full((2, kv, n + 9, dim), MARK, dtype=torch.float16, device="cuda")
        back = [whole[i, :, 4:4 + n].transpose(0, 1) for i in range(2)]
    for t in back:
        t.fill_(MARK)
    b.page_read_kv8(slots, *p, *back)
    b.check()
    keep = slots >= 0
    for rows, got in ((k, back[0]), (v, back[1])):
        want = values(*quantise(rows))
        want[~keep] = MARK
        assert same(got, want)
        # half a step of the block's scale, whose 127 / 64 holds the block's greatest
        # magnitude and with a quarter less (a step less for E5M2's subnormals) would not
        a = rows.double().unflatten(-1, (-1, BLOCK)).abs().amax(-1, keepdim=True)
        off = (got.double() - rows.double())[keep].unflatten(-1, (-1, BLOCK)).abs()
        assert (off <= (a * (5 / 4) / 127 + 2.0 ** -22).clamp(min=0)[keep] / 2).all()
    if layout == "packed":
        for i in (0, 2, 4, 5):
            assert (whole[:, i * kv * dim:(i + 1) * kv * dim] == MARK).all()
    elif layout == "heads":
        assert (whole[:, :, :4] == MARK).all() and (whole[:, :, 4 + n:] == MARK).all()


def test_every_number_against_every_scale():
    """All finite fp16 numbers under every scale that holds them: each block's first number
    brings the scale, the others are the numbers in order."""
    b = block(2, 1, 64)
    every = torch.arange(0x7c00, dtype=torch.int16, device="cuda").view(torch.float16)
    every = torch.cat((every, -every))
    for s in E5M2.tolist():
        top = torch.tensor(s * 127 / 64, dtype=torch.float64).clamp(max=65504).half().double()
        if top > s * 127 / 64:       # (rounded up: the next smaller fp16 number)
            top = torch.nextafter(top.half(), torch.tensor(0.0, dtype=torch.float16)).double()
        if top == 0:
            continue
        x = every[every.double().abs() <= top]
        x = torch.cat((x, x.new_zeros(-x.numel() % 31))).view(-1, 31)
        x = torch.cat((torch.full_like(x[:, :1], float(top)), x), 1)
        x = torch.cat((x, x.new_zeros((x.shape[0] % 2, 32)))).view(-1, 1, 64)
        n = x.shape[0]
        p = pools(-(-n // 128), 1, 128, 64)
        slots = torch.arange(n, device="cuda")
        b.page_append_kv8(x, -x, slots, *p)
        check_append(x, -x, slots, p)
    b.check()


def test_every_scale_boundary():
    """Every fp16 number as its block's greatest magnitude."""
    b = block(2, 1, 128)
    x = torch.zeros((0x7c00 // 4, 1, 128), dtype=torch.float16, device="cuda")
    x[:, 0, 5::32] = torch.arange(0x7c00, dtype=torch.int16, device="cuda").view(torch.float16).view(-1, 4)
    x[:, 0, 6::32] = -x[:, 0, 5::32] / 2
    p = pools(-(-x.shape[0] // 128), 1, 128, 128)
    slots = torch.arange(x.shape[0], device="cuda")
    b.page_append_kv8(x, -x, slots, *p)
    b.check()
    check_append(x, -x, slots, p)


def test_blocks_that_are_not_finite_read_as_nan_and_stay_alone():
    b = block(4, 2, 128)
    x = torch.randn((9, 2, 128), device="cuda").half()
    y = x.clone()
    for i, bad in enumerate((float("nan"), float("inf"), -float("inf"))):
        x[i, 0, 40 + i] = bad
        y[3 + i, 1, 127 - 31 * i] = bad
    x[7] = 0.0
    slots = torch.arange(9, device="cuda") + 3
    p = pools(1, 2, 16, 128)
    b.page_append_kv8(x, y, slots, *p)
    check_append(x, y, slots, p)
    back = [torch.full_like(x, MARK) for _ in range(2)]
    b.page_read_kv8(slots, *p, *back)
    b.check()
    for rows, got in ((x, back[0]), (y, back[1])):
        assert same(got, values(*quantise(rows)))
        assert got.isnan().sum().item() == 3 * BLOCK
    assert (back[0][7] == 0).all()


def test_read_of_every_code_and_scale():
    """All 256 codes under all 256 scale bytes, as fp16 holds the products."""
    b = block(2, 1, 64)
    code = torch.arange(256, device="cuda", dtype=torch.uint8).view(8, 32)
    p = pools(1024 // 16, 1, 16, 64)
    c, s = by_slot(p[0]), by_slot(p[2])
    c = code.repeat(1, 2).repeat(128, 1, 1).view(1024, 1, 64)              # 8 rows a pair of bytes
    s = torch.arange(256, device="cuda", dtype=torch.uint8).view(128, 1, 2).repeat_interleave(8, 0)
    for pool, rows in zip(p, (c, c.flip(-1), s, s.flip(-1))):
        pool.view(torch.uint8).copy_(rows.view(64, 16, 1, -1).transpose(1, 2))
    out = [torch.empty((1024, 1, 64), dtype=torch.float16, device="cuda") for _ in range(2)]
    b.page_read_kv8(torch.arange(1024, device="cuda"), *p, *out)
    b.check()
    for got, codes, scales in ((out[0], c, s), (out[1], c.flip(-1), s.flip(-1))):
        assert same(got, values(codes, scales).half())


def test_slots_outside_the_pool_are_reported_and_left():
    b = block(4, 2, 64)
    k = torch.ones((4, 2, 64), dtype=torch.float16, device="cuda")
    whole = pools(6, 2, 16, 64)
    p = [t[1:5] for t in whole]
    slots = torch.tensor([64, 5, -2, 2 ** 40], device="cuda")
    b.page_append_kv8(k, k, slots, *p)
    with pytest.raises(blk.BlkError) as e:
        b.check()
    assert e.value.status == blk.BLK_ERR_PAGE
    for t, wide in zip(whole, (64, 64, 2, 2)):
        at = (by_slot(t) != FILL).any(-1).any(-1).nonzero().flatten().tolist()
        assert at == [16 + 5], wide
    rows = [torch.full_like(k, MARK) for _ in range(2)]
    b.page_read_kv8(slots, *p, *rows)
    with pytest.raises(blk.BlkError) as e:
        b.check()
    assert e.value.status == blk.BLK_ERR_PAGE
    for r in rows:
        # (1 = 102.4 steps of the scale 0.625: 102 of them)
        assert same(r[1], values(*quantise(k[1]))) and (r[[0, 2, 3]] == MARK).all()


def test_read_of_one_slot_many_times_and_rows_in_any_order():
    b = block(4, 2, 64)
    x = torch.randn((40, 2, 64), device="cuda").half()
    p = pools(3, 2, 16, 64)
    b.page_append_kv8(x, x * 3, torch.arange(40, device="cuda"), *p)
    slots = torch.randint(0, 40, (1000,), device="cuda")
    out = [torch.empty((1000, 2, 64), dtype=torch.float16, device="cuda") for _ in range(2)]
    b.page_read_kv8(slots, *p, *out)
    b.check()
    for got, rows in zip(out, (x, x * 3)):
        assert same(got, values(*quantise(rows))[slots])


def test_a_captured_graph_takes_new_rows_and_slots():
    b = block(4, 2, 128)
    k, v = (torch.zeros((50, 2, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    slots = torch.zeros(50, dtype=torch.int64, device="cuda")
    p = pools(9, 2, 16, 128)
    out = [torch.zeros_like(k) for _ in range(2)]
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        b.page_append_kv8(k, v, slots, *p, stream=s)
        b.page_read_kv8(slots, *p, *out, stream=s)
    for seed in range(3):
        torch.manual_seed(seed)
        k.copy_(torch.randn(k.shape, device="cuda"))
        v.copy_(torch.randn(v.shape, device="cuda"))
        slots.copy_(torch.randperm(144, device="cuda")[:50])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        b.check()
        for got, rows in zip(out, (k, v)):
            assert same(got, values(*quantise(rows)))


def test_argument_errors():
    b = block(4, 2, 64)
    k, v = (torch.full((3, 2, 64), MARK, dtype=torch.float16, device="cuda") for _ in range(2))
    slots = torch.arange(3, device="cuda")
    p = pools(4, 2, 16, 64)
    st = torch.cuda.current_stream().cuda_stream
    P = [t.data_ptr() for t in p]
    S, A, N = blk.BLK_ERR_SHAPE, blk.BLK_ERR_ALIGN, blk.BLK_ERR_NULL

    def append(expect, h=b.handle, k=k.data_ptr(), v=v.data_ptr(), rs=128, hs=64, sm=slots.data_ptr(),
               n=3, page=16, pages=4, pool=P):
        q = blk.BlkKv8Pool(*pool) if pool else None
        assert blk.blk_page_append_kv8(h, k, v, rs, hs, sm, n, page, pages, q, st) == expect

    def read(expect, h=b.handle, k=k.data_ptr(), v=v.data_ptr(), rs=128, hs=64, sm=slots.data_ptr(),
             n=3, page=16, pages=4, pool=P):
        q = blk.BlkKv8Pool(*pool) if pool else None
        assert blk.blk_page_read_kv8(h, sm, n, page, pages, q, k, v, rs, hs, st) == expect

    for call in (append, read):
        for kw in (dict(h=None), dict(k=None), dict(v=None), dict(sm=None), dict(pool=None),
                   *(dict(pool=[*P[:i], None, *P[i + 1:]]) for i in range(4))):
            call(N, **kw)
        for kw in (dict(k=k.data_ptr() + 2), dict(v=v.data_ptr() + 8), dict(sm=slots.data_ptr() + 4),
                   dict(rs=132), dict(hs=65),
                   *(dict(pool=[*P[:i], P[i] + 8, *P[i + 1:]]) for i in range(4))):
            call(A, **kw)
        for kw in (dict(n=0), dict(n=(1 << 20) + 1), dict(page=48), dict(pages=0), dict(pages=1 << 31),
                   dict(rs=-128)):
            call(S, **kw)
    for kw in (dict(rs=0), dict(hs=0), dict(rs=64, hs=64), dict(rs=120, hs=64), dict(rs=64, hs=128)):
        read(S, **kw)
    torch.cuda.synchronize()
    assert (k == MARK).all() and all((t.view(torch.uint8) == FILL).all() for t in p)
    f = k.float()
    for i, bad in enumerate((f, k[:2], k.cpu(), k.transpose(1, 2))):
        with pytest.raises(blk.BlkError) as e:
            b.page_append_kv8(bad, v, slots, *p)
        assert e.value.status == S, i
        with pytest.raises(blk.BlkError) as e:
            b.page_read_kv8(slots, *p, v, bad)
        assert e.value.status == S, i
    for i in range(4):
        for bad in (p[i].view(torch.int8), p[i][:-1], p[i].cpu(), p[i].transpose(1, 2)):
            if i == 0 and bad.shape[0] == 3:
                continue           # (the first pool's shape is the others')
            with pytest.raises(blk.BlkError) as e:
                b.page_append_kv8(k, v, slots, *[bad if j == i else p[j] for j in range(4)])
            assert e.value.status == S
    with pytest.raises(blk.BlkError):
        b.page_append_kv8(k, v, slots.int(), *p)
    with pytest.raises(blk.BlkError):
        b.page_append_kv8(k, v.transpose(0, 1).contiguous().transpose(0, 1), slots, *p)
