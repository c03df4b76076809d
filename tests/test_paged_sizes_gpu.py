"""GPU tests of the attention's schedule at sizes that take its other branches: more
sequences than a thread of the many-row kernel each, and a line of tiles past 2^20, whose
ranges are formed in 64 bits."""
import math
import random

import pytest
import torch

from paged_reference import U16, Batch
from test_paged_gpu import MARK, block, check_rows, run_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,heads,kv,dim", [(385, 12, 2, 128), (700, 16, 16, 64),
                                               (4096, 4, 2, 64)])
def test_many_rows_of_many_sequences(seqs, heads, kv, dim):
    """A few tokens each, one of them a chunk, some idle."""
    rng = random.Random(seqs)
    hist = [rng.randint(0, 70) for _ in range(seqs)]
    new = [rng.choice([0, 1, 1, 2, 3]) for _ in range(seqs)]
    new[seqs // 2] = 40
    hist[seqs - 1], new[seqs - 1] = 900, 3
    x = Batch(heads, kv, dim, 16, hist, new, seed=61, pad_rows=2)
    out, b = run_attention(x)
    b.check()
    check_rows(x, out)


@pytest.mark.parametrize("slots,top,tile,head", [(1030, 1, 64, 1), (2061, 40, 128, 3)])
def test_a_line_of_more_than_2_20_tiles(slots, top, tile, head):
    """4096 sequences over the same pages (queries of their own), 16 kv heads: every row, in
    units inside one CTA and in cut ones."""
    B, kv, dim, page = 4096, 16, 64, 64
    assert B * kv * (-(-slots // tile) + head) > 1 << 20
    gen = torch.Generator("cuda")
    gen.manual_seed(62)
    n_pages = -(-slots // page)
    k, v = (torch.randn((n_pages, kv, page, dim), generator=gen, device="cuda").half()
            for _ in range(2))
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
    b.attn_paged(d, q, k, v, out, ws)
    b.check()
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), more)
    last = lens[seq] + torch.arange(n, device="cuda") - start[seq]
    seen = torch.arange(n_pages * page, device="cuda") <= last[:, None]
    for h in range(kv):        # (the bound of tests/paged_reference.py)
        kh, vh = (t[:, h].reshape(-1, dim).double() for t in (k, v))
        s = (q[:, h].double() @ kh.T / math.sqrt(dim)).masked_fill(~seen, -math.inf)
        e = torch.exp(s - s.amax(-1, keepdim=True))
        l = e.sum(-1, keepdim=True)
        want, A = e / l @ vh, e / l @ vh.abs()
        sub = seen.sum(-1, keepdim=True) * 2.0 ** -25 * vh.abs().max() / l
        bound = (U16 + 2.0 ** -13) * A + sub + U16 * want.abs() + 2.0 ** -25
        worst = ((out[:, h].double() - want).abs() / bound).amax(-1)
        assert worst.max().item() <= 1.0, f"head {h}, row {worst.argmax().item()}"
