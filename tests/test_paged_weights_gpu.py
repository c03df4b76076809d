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



@pytest.mark.parametrize("top", [1, 60])
@pytest.mark.parametrize("prefix", [0, 8192])
def test_a_slot_far_above_all_others_is_the_result(top, prefix):
    """Scores of 10^7 and more, whose fp32 values are whole numbers apart: weights stay in
    fp16's range, and the row is that slot's V (its weight and the result rounded once each,
    U16 of |V|; its exponential and their quotient in fp32).  The slot is another one, and of another
    score, in every sequence and kv head."""
    hist = [prefix + 200 + 37 * (i % 5) for i in range(60)]
    x = Batch(12, 2, 128, 64, hist, [top] + [1] * 59, seed=44, prefix=prefix)
    x.k_pages[~x.k_pages.isnan()] = 0
    x.q[..., 0] = 30000
    want = torch.empty_like(x.q)
    r0 = 0
    for b, (have, more) in enumerate(zip(x.hist, x.new)):
        for g in range(2):
            at = prefix + 3 * b + g
            pg = int(x.table[b, at // 64])
            x.k_pages[pg, g, at % 64, 0] = 8000 + 199 * b + 64 * g
            want[r0:r0 + more, g * 6:g * 6 + 6] = x.v_pages[pg, g, at % 64]
        r0 += more
    out, b = run_attention(x)
    b.check()
    off = (out.double() - want.double()).abs()
    assert (off <= (2 * U16 + 2.0 ** -13) * want.double().abs() + 2.0 ** -25).all()


@pytest.mark.parametrize("step", [60, 94, 200, -94])
@pytest.mark.parametrize("k0", [12000, 18000, 25000])
@pytest.mark.parametrize("top,prefix", [(1, 0), (60, 0), (1, 8192)])
def test_large_scores_that_rise_from_tile_to_tile(top, prefix, k0, step):
    """Scores of 3 - 7 10^7 that grow or fall by some e-folds from one 128 slots to the next:
    their weights are rough (fp32 holds such scores to 2 - 8), but a row stays between the least and
    the greatest of V, weights and their sum being of the same exponentials (each weight,
    and the result, rounded once)."""
    hist = [prefix + 900 + 37 * (i % 5) for i in range(60)]
    x = Batch(12, 2, 128, 128, hist, [top] + [1] * 59, seed=45, prefix=prefix)
    seen = ~x.k_pages.isnan()
    x.k_pages[seen] = 0
    x.v_pages[seen] = 1 + x.v_pages[seen].abs().clamp(max=1)
    x.q[..., 0], x.q[..., 1] = 30000, 1
    for b, (have, more) in enumerate(zip(x.hist, x.new)):
        for j in range(-(-(have + more) // 128)):
            pg = int(x.table[b, j])
            x.k_pages[pg, :, :, 0] = torch.where(seen[pg, :, :, 0], k0, x.k_pages[pg, :, :, 0])
            x.k_pages[pg, :, :, 1] = torch.where(seen[pg, :, :, 1], 94 * 100 + step * (j - 60),
                                                 x.k_pages[pg, :, :, 1])
    out, b = run_attention(x)
    b.check()
    got = out[:x.n].double()
    assert got.min().item() >= 1 - 2 * U16 - 2.0 ** -13 and got.max().item() <= 2 + 4 * U16 + 2.0 ** -12
