"""GPU tests of rows over an 8-bit paged cache whose scores fall from slot to slot beside
rows whose scores are very large, or not finite: each row keeps to its own bound."""
import math

import pytest
import torch

from kv8_reference import in_8_bits
from paged_reference import U16, Batch, gather
from test_kv8_attn_gpu import run8

pytestmark = pytest.mark.gpu
LARGE, FALL = 0, 40             # columns: of the large scores, of the falling ones


def falling(heads, kv, dim, top, value, tiles=80, step=2.0):
    """One sequence, and a batch of as many copies of it (over the same pages) as give every CTA
    a whole one.  Scores of every third head are value * k / sqrt(dim) with k = 8000 in every
    slot and 16000 in slot 5; those of the others fall by `step` (log2 units) a tile of the
    few-row kernel, 160 in all, and what the other columns add is a tenth of a unit.  K's 8
    bits move a score by 160 * 1.25 / 254 = 0.8 at most, so no tile is 4 below the one before."""
    wide = top * heads // kv > 16
    tile = (64 if dim == 128 else 128) << wide
    x = Batch(heads, kv, dim, 64, [tiles * tile - top], [top], seed=50, extra_pages=0)
    n = tiles * tile
    k = torch.randn((n, kv, dim), device="cuda") * 0.1
    k[:, :, :32] = 0                                     # (LARGE has its block to itself)
    k[..., LARGE] = 8000
    k[5, :, LARGE] = 16000
    fall = -step / tile * math.log(2) * math.sqrt(dim) / 16
    k[..., FALL] = (fall * torch.arange(n, device="cuda"))[:, None]
    where = x.table[0, :n // 64].long()
    x.k_pages[where] = k.half().view(n // 64, 64, kv, dim).transpose(1, 2)
    large = torch.arange(heads, device="cuda") % 3 == 1
    x.q[..., LARGE] = 0
    x.q[..., FALL] = 16
    x.q[:, large, LARGE] = value
    in_8_bits(x)
    return x, large, n


def copies(x, B):
    x.hist, x.new = x.hist * B, x.new * B
    x.n = x.rows = x.n * B
    x.row_start = torch.arange(B + 1, device="cuda") * x.new[0]
    x.lens, x.table, x.q = x.lens.repeat(B), x.table.repeat(B, 1), x.q.repeat(B, 1, 1)
    return x


def reference(x, n, skip):
    """(out, bound) of the one sequence.  The bound is that of paged_reference.attention but for
    the falling column, whose terms are not of unit scale: a score's sum of dim products, its
    factor log2(e) / sqrt(dim) and the exponent's own rounding are off by (dim + 2) 2^-24 of
    that term, e, and move the numerator by sum p e |v| and the denominator by sum p e."""
    table = x.table[0, :n // 64]
    k, v = (gather(p, table, n) for p in (x.k_pages, x.v_pages))
    top, G = x.new[0], x.heads // x.kv
    out = torch.zeros((top, x.heads, x.dim), dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(out)
    seen = torch.arange(n, device="cuda") <= x.hist[0] + torch.arange(top, device="cuda")[:, None]
    for h in range(x.heads):
        if skip[h]:
            continue
        q, kh, vh = x.q[:top, h].double(), k[h // G], v[h // G]
        s = (q @ kh.T / math.sqrt(x.dim)).masked_fill(~seen, -math.inf)
        e = torch.exp(s - s.amax(-1, keepdim=True))
        l = e.sum(-1, keepdim=True)
        p = e / l
        off = (x.dim + 2) * 2.0 ** -24 * (q[:, FALL, None] * kh[:, FALL]).abs() / math.sqrt(x.dim)
        out[:, h] = p @ vh
        A = p @ vh.abs()
        lost = n * 2.0 ** -25 * vh.abs().max() / l
        bound[:, h] = ((U16 + 2.0 ** -13) * A + lost + U16 * out[:, h].abs() + 2.0 ** -25 +
                       (p * off) @ vh.abs() + (p * off).sum(-1, keepdim=True) * A)
    return out, bound


# 1 - 4 tiles of eight rows, of 128 and of 64 columns; many rows
SHAPES = [(12, 2, 128, 1), (12, 2, 128, 2), (12, 2, 128, 4), (16, 4, 128, 8), (16, 4, 64, 1),
          (16, 4, 64, 3), (16, 4, 64, 6), (16, 4, 64, 8), (12, 2, 128, 40)]


@pytest.mark.parametrize("heads,kv,dim,top", SHAPES)
@pytest.mark.parametrize("value", [30000.0, -30000.0, math.inf, -math.inf, math.nan])
def test_falling_scores_beside_large_ones(heads, kv, dim, top, value):
    x, large, n = falling(heads, kv, dim, top, value)
    want, bound = reference(x, n, large)
    slot5 = x.v_pages[x.table[0, 0].long(), :, 5].double()
    v_max = x.v_pages[~x.v_pages.isnan()].abs().max().item()
    B = 456 // kv if top * heads // kv <= 16 else 152 // kv
    out, b = run8(copies(x, B))
    b.check()
    got = out.view(B, top, heads, dim).double()
    worst = ((got - want).abs() / bound.clamp(min=1e-30))[:, :, ~large].amax().item()
    assert worst <= 1.0, f"{worst:.3g} of the bound"
    if value == 30000.0:                 # slot 5 is far above all others
        v = slot5.repeat_interleave(heads // kv, 0)[large]
        assert ((got[:, :, large] - v).abs() <= (2 * U16 + 2.0 ** -13) * v.abs() + 2.0 ** -25).all()
    elif math.isfinite(value):           # it is far below them: a mean of the others
        assert (got[:, :, large].abs() <= v_max * (1 + 2 * U16 + 2.0 ** -13)).all()
    elif math.isnan(value) or value > 0:
        assert got[:, :, large].isnan().all()
