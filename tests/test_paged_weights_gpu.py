"""GPU tests of small softmax weights: rows in which one slot outweighs all others by up
to e^17 and hides nothing of them (its own values are small), against a 64-bit
evaluation whose bound has no room for weights that are lost."""
import math

import pytest
import torch

from paged_reference import U16, Batch, gather
from test_paged_gpu import block, prefix_launches, run_attention

pytestmark = pytest.mark.gpu
# The kernels form a weight as 2^kFew (few rows) or 2^kMany (many rows, a prefix's own
# launch) times exp(s - max) before it is rounded to fp16: below 2^-14 of that it is off by
# half a step, 2^-25.
K_FEW, K_MANY = 14, 7


def with_sink(x, at, nats):
    """All scores 0 but that of slot `at` of every sequence, which is `nats`; values of 1
    and more but there, where they are a hundredth."""
    for pool in (x.k_pages, x.v_pages):
        seen = ~pool.isnan()
        pool[seen] = 0 if pool is x.k_pages else pool[seen].abs() + 1
    x.q[..., 0] = 8
    for b, (have, more) in enumerate(zip(x.hist, x.new)):
        if have > at:
            pg = int(x.table[b, at // x.page])
            if x.k_pages[pg, 0, at % x.page, 0] == 0:      # (a prefix's page: once)
                x.k_pages[pg, :, at % x.page, 0] = nats * math.sqrt(x.dim) / 8
                x.v_pages[pg, :, at % x.page] /= 100
    return x


def check_weights(x, out, factor):
    """With p the weights, A = sum p |v| and l the sum of exp(s - max): weights and result
    are rounded to fp16 (U16 A, 2^-25 / 2^factor / l absolutely for the weights; U16 |out|,
    2^-25), scores (here at most 18), exponentials and sums are fp32 (2^-13 A)."""
    r0 = 0
    for b, (have, more) in enumerate(zip(x.hist, x.new)):
        n = have + more
        k, v = (gather(p, x.table[b, :-(-n // x.page)], n) for p in (x.k_pages, x.v_pages))
        seen = torch.arange(n, device="cuda") <= have + torch.arange(more, device="cuda")[:, None]
        for h in range(x.heads):
            kh, vh = (t[h // (x.heads // x.kv)] for t in (k, v))
            s = x.q[r0:r0 + more, h].double() @ kh.T / math.sqrt(x.dim)
            s = s.masked_fill(~seen, -math.inf)
            e = torch.exp(s - s.amax(-1, keepdim=True))
            l = e.sum(-1, keepdim=True)
            want, A = e / l @ vh, e / l @ vh.abs()
            lost = seen.sum(-1, keepdim=True) * 2.0 ** (-25 - factor) * vh.abs().max() / l
            bound = (U16 + 2.0 ** -13) * A + lost + U16 * want.abs() + 2.0 ** -25
            worst = ((out[r0:r0 + more, h].double() - want).abs() / bound).max().item()
            assert worst <= 1.0, f"sequence {b}, head {h}: {worst:.3g} of the bound"
        r0 += more


@pytest.mark.parametrize("nats", [9.0, 12.0, 15.0, 17.4])
@pytest.mark.parametrize("at", [0, 70, 8000])
@pytest.mark.parametrize("heads,kv,dim,top", [(12, 2, 128, 1), (12, 2, 128, 5), (4, 2, 64, 2)])
def test_few_rows(heads, kv, dim, top, at, nats):
    x = Batch(heads, kv, dim, 64, [32000, 90, 9000, 4], [1, top, top, 1], seed=41)
    x = with_sink(x, at, nats)
    out, b = run_attention(x)
    b.check()
    check_weights(x, out, K_FEW)


@pytest.mark.parametrize("nats", [9.0, 12.0, 15.0, 17.4])
@pytest.mark.parametrize("at", [0, 140, 5000])
@pytest.mark.parametrize("heads,kv,dim", [(12, 2, 128), (16, 16, 64)])
def test_many_rows(heads, kv, dim, at, nats):
    x = Batch(heads, kv, dim, 32, [12000, 200, 6001], [50, 1, 300], seed=42)
    x = with_sink(x, at, nats)
    out, b = run_attention(x)
    b.check()
    check_weights(x, out, K_MANY)


@pytest.mark.parametrize("nats", [9.0, 15.0, 17.4])
@pytest.mark.parametrize("at", [0, 3000, 8200])
@pytest.mark.parametrize("top", [1, 40])
def test_shared_prefix(top, at, nats):
    """The sink in the prefix's own launch, or among each sequence's own slots behind it."""
    hist = [8192 + (0, 300, 9)[i % 3] for i in range(60)]
    x = Batch(12, 2, 128, 64, hist, [1 + i % top for i in range(60)], seed=43, prefix=8192)
    x = with_sink(x, at, nats)
    (out, b), n = prefix_launches(block(12, 2, 128), lambda: run_attention(x))
    b.check()
    assert n == 1
    check_weights(x, out, K_MANY)

