"""GPU tests of the 8-bit caches' attention at sizes that take the schedule's other branches,
of tensors whose strides of a dimension of size one mean nothing, and of the operators run
together, captured once and replayed over growing lengths."""
import math
import random

import pytest
import torch

import decode_qwen2_block_gb300 as blk
from kv8_reference import BLOCK, in_8_bits, quantise, same, values
from paged_reference import U16, Batch, attention
from test_kv8_attn_gpu import run8
from test_paged_gpu import MARK, block, check_rows

pytestmark = pytest.mark.gpu
E5 = torch.float8_e5m2


def _pools(n_pages, kv, page, dim):
    def make(last):
        return torch.zeros((n_pages, kv, page, last), dtype=torch.uint8, device="cuda")
    return [make(dim), make(dim), make(dim // BLOCK).view(E5), make(dim // BLOCK).view(E5)]


@pytest.mark.parametrize("seqs,heads,kv,dim", [(385, 12, 2, 128), (700, 16, 16, 64),
                                               (4096, 4, 2, 64)])
@pytest.mark.parametrize("top", [1, 4, 40])
def test_many_sequences(seqs, heads, kv, dim, top):
    """A few tokens each, one of them a chunk, some idle."""
    rng = random.Random(seqs)
    hist = [rng.randint(0, 70) for _ in range(seqs)]
    new = [rng.choice([0, 1, 1, min(2, top), min(3, top)]) for _ in range(seqs)]
    new[seqs // 2] = top
    hist[seqs - 1], new[seqs - 1] = 900, min(3, top)
    x = in_8_bits(Batch(heads, kv, dim, 16, hist, new, seed=61, pad_rows=2))
    out, b = run8(x)
    b.check()
    check_rows(x, out)


@pytest.mark.parametrize("slots,top,head", [(1930, 1, 1), (2061, 40, 3)])
def test_a_line_of_more_than_2_20_tiles(slots, top, head):
    """4096 sequences over the same pages (queries of their own), 16 kv heads of 64 columns
    (tiles of 128 slots): every row, in units inside one CTA and in cut ones."""
    B, kv, dim, page = 4096, 16, 64, 64
    assert B * kv * (-(-slots // 128) + head) > 1 << 20
    gen = torch.Generator("cuda")
    gen.manual_seed(62)
    n_pages = -(-slots // page)
    raw = [torch.randn((n_pages, kv, page, dim), generator=gen, device="cuda").half() for _ in range(2)]
    (kc, ks), (vc, vs) = (quantise(t) for t in raw)
    k, v = values(kc, ks), values(vc, vs)
    new = [1] * B
    new[1000] = top
    n = sum(new)
    q = torch.randn((n, kv, dim), generator=gen, device="cuda").half()
    start = torch.tensor([0] + new, device="cuda").cumsum(0)
    more = torch.tensor(new, device="cuda")
    lens = slots - more                                      # every sequence ends at `slots`
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    b = block(kv, kv, dim)
    d = b.paged_batch(start, lens, table, n, page, n_pages, top, slots)
    ws = torch.full((b.attn_paged_workspace_bytes(n, B),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((n, kv, dim), MARK, dtype=torch.float16, device="cuda")
    b.attn_paged_kv8(d, q, kc, vc, ks.view(E5), vs.view(E5), out, ws)
    b.check()
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), more)
    last = lens[seq] + torch.arange(n, device="cuda") - start[seq]
    seen = torch.arange(n_pages * page, device="cuda") <= last[:, None]
    for h in range(kv):        # (the bound of tests/paged_reference.py)
        kh, vh = (t[:, h].reshape(-1, dim) for t in (k, v))
        s = (q[:, h].double() @ kh.T / math.sqrt(dim)).masked_fill(~seen, -math.inf)
        e = torch.exp(s - s.amax(-1, keepdim=True))
        l = e.sum(-1, keepdim=True)
        want, A = e / l @ vh, e / l @ vh.abs()
        sub = seen.sum(-1, keepdim=True) * 2.0 ** -25 * vh.abs().max() / l
        bound = (U16 + 2.0 ** -13) * A + sub + U16 * want.abs() + 2.0 ** -25
        worst = ((out[:, h].double() - want).abs() / bound).amax(-1)
        assert worst.max().item() <= 1.0, f"head {h}, row {worst.argmax().item()}"


@pytest.mark.parametrize("heads,kv,dim", [(12, 2, 128), (4, 2, 64)])
def test_one_row_out_of_head_major_tensors(heads, kv, dim):
    x = in_8_bits(Batch(heads, kv, dim, 64, [300], [1], seed=51))
    q = torch.empty((heads, 1, dim), dtype=torch.float16, device="cuda").transpose(0, 1)
    q.copy_(x.q)
    x.q = q
    out = torch.full((heads, 1, dim), MARK, dtype=torch.float16, device="cuda").transpose(0, 1)
    assert q.stride(0) == out.stride(0) == dim
    _, b = run8(x, out=out)
    b.check()
    check_rows(x, out)


@pytest.mark.parametrize("n,kv", [(1, 2), (5, 1), (1, 1)])
def test_rows_of_differing_strides_where_they_mean_nothing(n, kv):
    dim = 64
    k = torch.randn((n, kv, dim), device="cuda").half()
    packed = torch.randn((n, 6, kv, dim), device="cuda").half()
    v = packed[:, 3] if n == 1 else packed[:, 0].contiguous()
    k = k.as_strided((n, kv, dim), (k.stride(0) if n > 1 else 3, 5 if kv == 1 else dim, 1))
    p = _pools(3, kv, 16, dim)
    slots = torch.tensor([40, 3, 17, 5, 0][:n], device="cuda")
    b = block(kv * 2, kv, dim)
    b.page_append_kv8(k, v, slots, *p)
    back = [torch.zeros_like(t) for t in (k, v)]
    back[0] = back[0].as_strided((n, kv, dim), k.stride())
    b.page_read_kv8(slots, *p, *back)
    b.check()
    for got, rows in zip(back, (k, v)):
        assert same(got, values(*quantise(rows)))


def test_the_same_rows_for_every_slot():
    """A broadcast row (stride 0) is appended to many slots; rows over each other are not read to."""
    b = block(4, 2, 64)
    row = torch.randn((1, 2, 64), device="cuda").half()
    p = _pools(3, 2, 16, 64)
    slots = torch.randperm(48, device="cuda")
    many = row.expand(48, 2, 64)
    b.page_append_kv8(many, many, slots, *p)
    out = [torch.zeros((48, 2, 64), dtype=torch.float16, device="cuda") for _ in range(2)]
    b.page_read_kv8(slots, *p, *out)
    b.check()
    for got in out:
        assert same(got, values(*quantise(many)))
    with pytest.raises(blk.BlkError) as e:
        b.page_read_kv8(slots, *p, torch.zeros_like(row).expand(48, 2, 64), torch.zeros_like(row).expand(48, 2, 64))
    assert e.value.status == blk.BLK_ERR_SHAPE


@pytest.mark.parametrize("heads,kv,dim,page", [(12, 2, 128, 16), (4, 2, 64, 64)])
def test_the_operators_together_in_one_graph(heads, kv, dim, page):
    """Plan, append, attention and read of a step, captured once and replayed as sequences grow
    by drafts and tokens: every row against its definition over what the cache has been given."""
    b = block(heads, kv, dim)
    B, rows, cap = 3, 7, 160
    blocks = -(-cap // page)
    i64 = dict(dtype=torch.int64, device="cuda")
    lens, news, start = torch.zeros(B, **i64), torch.zeros(B, **i64), torch.zeros(B + 1, **i64)
    slots, pos, used = torch.zeros(rows, **i64), torch.zeros(rows, **i64), torch.zeros(1, **i64)
    free = torch.zeros(B, dtype=torch.int32, device="cuda")
    table = torch.full((B, blocks), -1, dtype=torch.int32, device="cuda")
    p = _pools(B * blocks, kv, page, dim)
    q = torch.zeros((rows, heads, dim), dtype=torch.float16, device="cuda")
    k, v, kb, vb = (torch.zeros((rows, kv, dim), dtype=torch.float16, device="cuda") for _ in range(4))
    out = torch.zeros_like(q)
    ws = torch.empty(b.attn_paged_workspace_bytes(rows, B, prefix=False), dtype=torch.uint8, device="cuda")
    d = b.paged_batch(start, lens, table, rows, page, B * blocks, 4, cap)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        b.page_plan(page, lens, news, free, table, start, slots, pos, used, stream=s)
        b.page_append_kv8(k, v, slots, *p, stream=s)
        b.attn_paged_kv8(d, q, *p, out, ws, stream=s)
        b.page_read_kv8(slots, *p, kb, vb, stream=s)
    ids = list(range(B * blocks))
    held = [[torch.zeros((kv, 0, dim), dtype=torch.float64, device="cuda") for _ in range(2)]
            for _ in range(B)]
    rng = random.Random(3)
    for step in range(40):
        new = [rng.choice([0, 1, 1, 4]) for _ in range(B)]
        while sum(new) > rows:
            new[new.index(4)] = 1
        n = sum(new)
        torch.manual_seed(step)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, device="cuda"))
        news.copy_(torch.tensor(new))
        free.copy_(torch.tensor((ids + [-1] * B)[:B], dtype=torch.int32))
        kb.fill_(MARK)
        vb.fill_(MARK)
        out.fill_(MARK)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        b.check()
        del ids[:int(used)]
        want_k, want_v = values(*quantise(k)), values(*quantise(v))
        assert same(kb[:n], want_k[:n]) and same(vb[:n], want_v[:n])
        assert (kb[n:] == MARK).all() and (out[n:] == MARK).all()
        at = 0
        for i, t in enumerate(new):
            have = held[i][0].shape[1]
            if t:
                held[i] = [torch.cat((old, w[at:at + t].transpose(0, 1)), 1)
                           for old, w in zip(held[i], (want_k, want_v))]
                want, bound = attention(q[at:at + t], *held[i], have)
                assert ((out[at:at + t].double() - want).abs() <= bound).all(), (step, i)
            at += t
        lens.copy_(torch.tensor([h[0].shape[1] for h in held]))
