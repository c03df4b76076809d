"""Attention over a paged cache in 64 bits, row by row from the definition, and
the bound that a kernel's fp16 result has to keep against it."""
from __future__ import annotations

import math

import torch

U16 = 2.0 ** -11      # unit roundoff of fp16


def gather(pool, pages, n):
    """Slots [0, n) of a sequence: [heads, n, dim] in 64 bits."""
    return pool[pages.long()].transpose(0, 1).flatten(1, 2)[:, :n].double()


def attention(q, k, v, have, window=0):
    """q [n, heads, dim], k/v [kv_heads, have + n, dim] -> (out, bound), both [n, heads, dim].

    The bound per element, with p the softmax weights, A = sum p |v| and l the sum
    of exp(s - max): the weights are rounded to fp16 (U16 A; those below 2^-14 by
    2^-25 absolutely, seen * 2^-25 max|v| / l), scores, exponentials and sums are
    fp32 (a score's error is at most dim 2^-24 sum |q k| / sqrt(dim), below 6e-5
    for unit-scale rows of 128; it moves numerator and denominator: 2^-13 A), and
    the result is rounded once (U16 |out|, 2^-25 where it is subnormal)."""
    n, heads, dim = q.shape
    kv = k.shape[0]
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    bound = torch.empty_like(out)
    col = torch.arange(k.shape[1], device=q.device)
    last = have + torch.arange(n, device=q.device)[:, None]
    seen = col <= last
    if window > 0:
        seen &= col > last - window
    some = seen.any(0)
    for h in range(heads):
        kh, vh = k[h // (heads // kv)], v[h // (heads // kv)]
        kh = torch.where(some[:, None], kh, torch.zeros_like(kh))
        vh = torch.where(some[:, None], vh, torch.zeros_like(vh))
        s = (q[:, h].double() @ kh.T / math.sqrt(dim)).masked_fill(~seen, -math.inf)
        e = torch.exp(s - s.amax(-1, keepdim=True))
        l = e.sum(-1, keepdim=True)
        p = e / l
        out[:, h] = p @ vh
        A = p @ vh.abs()
        sub = seen.sum(-1, keepdim=True) * 2.0 ** -25 * vh.abs().max() / l
        bound[:, h] = (U16 + 2.0 ** -13) * A + sub + U16 * out[:, h].abs() + 2.0 ** -25
    return out, bound


class Batch:
    """A ragged batch over pools of random pages: sequence b holds hist[b] slots and
    gets new[b] rows.  Every slot that no row sees holds `junk`, tables are filled
    with `unused` behind the last page."""

    def __init__(self, heads, kv, dim, page, hist, new, seed=0, prefix=0, pad_rows=0,
                 junk=math.nan, unused=-1, packed=False, extra_pages=3, n_pages=None,
                 device="cuda"):
        gen = torch.Generator(device)
        gen.manual_seed(seed)
        self.heads, self.kv, self.dim, self.page = heads, kv, dim, page
        self.hist, self.new, self.prefix_len = hist, new, prefix
        B, self.n = len(hist), sum(new)
        first = prefix // page
        need = [-(-(h + t) // page) for h, t in zip(hist, new)]
        own = [max(0, k - first) for k in need]
        count = first + sum(own)
        total = count + extra_pages if n_pages is None else n_pages
        ids = torch.randperm(total, generator=gen, device=device)[:count].to(torch.int32)
        if n_pages is not None:          # the last pages of a large pool are among them
            ids[-1] = total - 1 if not (ids == total - 1).any() else ids[-1]
        self.max_blocks = max(need + [1]) + 2
        self.table = torch.full((B, self.max_blocks), unused, dtype=torch.int32, device=device)
        at = first
        for b in range(B):
            self.table[b, :first] = ids[:first]
            self.table[b, first:first + own[b]] = ids[at:at + own[b]]
            at += own[b]
        self.prefix = ids[:first].contiguous() if prefix else None
        shape = (total, kv, page, dim)
        self.k_pages = torch.empty(shape, dtype=torch.float16, device=device)
        self.v_pages = torch.empty(shape, dtype=torch.float16, device=device)
        used = ids.long()
        if n_pages is None:
            self.k_pages.fill_(junk)
            self.v_pages.fill_(junk)
        for pool in (self.k_pages, self.v_pages):
            pool[used] = torch.randn((count, kv, page, dim), generator=gen, device=device).half()
        for b in range(B):               # slots behind the last one
            n = hist[b] + new[b]
            if n % page and need[b] > first:
                pg = int(self.table[b, n // page])
                self.k_pages[pg, :, n % page:] = junk
                self.v_pages[pg, :, n % page:] = junk
        rows = self.n + pad_rows
        width = heads * dim + (2 * kv * dim if packed else 0)
        self.q = torch.randn((rows, width), generator=gen, device=device).half()
        self.q = self.q[:, :heads * dim].unflatten(1, (heads, dim))
        self.lens = torch.tensor(hist, dtype=torch.int64, device=device)
        self.row_start = torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int64,
                                      device=device)
        self.rows = rows

    def descriptor(self, block, **kw):
        a = dict(max_new=max(self.new + [1]),
                 max_len=max([h + t for h, t in zip(self.hist, self.new)] + [1]),
                 prefix_pages=self.prefix)
        a.update(kw)
        return block.paged_batch(self.row_start, self.lens, self.table, self.rows, self.page,
                                 self.k_pages.shape[0], **a)

    def reference(self, window=0, skip=()):
        out = torch.zeros((self.rows, self.heads, self.dim), dtype=torch.float64, device=self.q.device)
        bound = torch.zeros_like(out)
        at = 0
        for b, (h, t) in enumerate(zip(self.hist, self.new)):
            if t and b not in skip:
                pages = self.table[b, :-(-(h + t) // self.page)]
                k, v = (gather(pool, pages, h + t) for pool in (self.k_pages, self.v_pages))
                out[at:at + t], bound[at:at + t] = attention(self.q[at:at + t], k, v, h, window)
            at += t
        return out, bound
