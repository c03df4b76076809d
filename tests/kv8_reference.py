"""The 8-bit form of a paged cache in 64 bits, from its definition, and batches over
such caches."""
from __future__ import annotations

import math

import torch

from paged_reference import Batch

BLOCK = 32
NAN_SCALE = 0x7f

# every finite, positive E5M2 number in ascending order, by the bytes 1 .. 123
E5M2 = torch.tensor([(b & 3) * 2.0 ** -16 if b < 4 else (4 + (b & 3)) * 2.0 ** ((b >> 2) - 17)
                     for b in range(1, 124)], dtype=torch.float64)


def scale_of(byte):
    """Scale bytes (uint8) as numbers, in 64 bits."""
    table = torch.zeros(256, dtype=torch.float64, device=byte.device)
    table[1:124] = E5M2.to(byte.device)
    table[124] = math.inf
    table[125:128] = math.nan
    table[128:] = -table[:128]
    return table[byte.long()]


def quantise(x):
    """fp16 [..., dim] -> (codes uint8 [..., dim], scale bytes uint8 [..., dim / 32]): the least
    E5M2 number s with 127 s / 64 >= the block's greatest magnitude, codes 64 x / s rounded
    to the nearest, ties to even (64-bit quotients of fp16 by 3-bit numbers are half way
    where the quotient is)."""
    b = x.double().unflatten(-1, (-1, BLOCK))
    a = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    # (127 s / 64 is exact)
    byte = torch.searchsorted(E5M2.to(x.device) * 127 / 64, a.masked_fill(bad, 0).contiguous()) + 1
    byte = torch.where(a > 0, byte, 0)
    s = scale_of(byte)
    c = torch.round(b.masked_fill(bad[..., None], 0) * 64 / torch.where(s > 0, s, 1.0)[..., None])
    assert c.abs().max() <= 127
    byte = torch.where(bad, NAN_SCALE, byte)
    return (c + 128).to(torch.uint8).flatten(-2), byte.to(torch.uint8)


def values(codes, scales):
    """What codes with scale bytes stand for, in 64 bits."""
    c = codes.double().unflatten(-1, (-1, BLOCK)) - 128
    return (c * (scale_of(scales) / 64)[..., None]).flatten(-2)


def same(a, b):
    """Equal values, NaN in the same places."""
    a, b = a.double(), b.double()
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))


def in_8_bits(x: Batch) -> Batch:
    """The batch over pools in 8 bits: codes and scales beside the fp16 pools, which become what
    they stand for.  (Of a NaN block's codes nothing is known: they are made to differ.)"""
    x.pools8 = []
    for name in ("k_pages", "v_pages"):
        pool = getattr(x, name)
        codes, scales = torch.empty(pool.shape, dtype=torch.uint8, device=pool.device), None
        scales = torch.empty((*pool.shape[:3], pool.shape[3] // BLOCK), dtype=torch.uint8,
                             device=pool.device)
        some = max(1, (1 << 24) // pool[0].numel())
        for i in range(0, pool.shape[0], some):
            codes[i:i + some], scales[i:i + some] = quantise(pool[i:i + some])
            v = values(codes[i:i + some], scales[i:i + some])
            assert same(v.half(), v)
            setattr(x, name, pool)
            pool[i:i + some] = v.half()
        nan = scales == NAN_SCALE
        if nan.any():
            at = codes.unflatten(-1, (-1, BLOCK))
            at[nan] = torch.arange(int(nan.sum()) * BLOCK, device=pool.device).to(torch.uint8).view(-1, BLOCK)
        x.pools8.append((codes, scales))
    (kc, ks), (vc, vs) = x.pools8
    e5 = torch.float8_e5m2
    x.pools8 = (kc, vc, ks.view(e5), vs.view(e5))
    return x
