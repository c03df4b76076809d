"""GPU tests of attention over 8-bit paged caches: the batches of the fp16 caches' tests,
against a 64-bit evaluation of the definition over the values that codes and scales stand
for (exact in fp16), within the bound that the roundings behind them give
(tests/paged_reference.py)."""
import random

import pytest
import torch

import decode_qwen2_block_gb300 as blk
from kv8_reference import NAN_SCALE, in_8_bits, quantise, values
from paged_reference import U16, Batch
from test_paged_gpu import HEADS, MARK, block, check_rows
from test_paged_weights_gpu import K_MANY, check_weights, with_sink

pytestmark = pytest.mark.gpu
# The few-row kernel forms a weight as 2^K8_FEW times exp(s - m) before it is rounded to
# fp16, with m at or below the row's maximum; the many-row kernel is the fp16 caches'.
K8_FEW = 10


def run8(x, window=0, out=None, stream=None, shift=0, **kw):
    b = block(x.heads, x.kv, x.dim, window)
    d = x.descriptor(b, **kw)
    if out is None:
        out = torch.full((x.rows, x.heads, x.dim), MARK, dtype=torch.float16, device="cuda")
    nb = b.attn_paged_workspace_bytes(x.rows, len(x.hist), prefix=d.prefix_len > 0)
    ws = torch.full((nb + 32,), 255, dtype=torch.uint8, device="cuda")     # NaN wherever it is read
    b.attn_paged_kv8(d, x.q, *x.pools8, out, ws[shift:shift + nb], stream=stream)
    return out, b


def batch8(*a, **kw):
    return in_8_bits(Batch(*a, **kw))


@pytest.mark.parametrize("heads,kv,dim", HEADS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_decode(heads, kv, dim, page):
    """One token per sequence, histories from none to many tiles, an idle sequence, NaN
    blocks in every slot past a sequence's last and in every other page."""
    hist = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 1000, 0, 300]
    new = [1] * len(hist)
    new[-1] = 0
    x = batch8(heads, kv, dim, page, hist, new, seed=page + heads, pad_rows=3, packed=page == 32)
    out, b = run8(x)
    b.check()
    check_rows(x, out)


@pytest.mark.parametrize("heads,kv,dim", HEADS)
@pytest.mark.parametrize("top", [2, 4, 9])
def test_few_new_tokens(heads, kv, dim, top):
    rng = random.Random(top)
    hist = [rng.choice([0, 3, 62, 63, 64, 129, 700]) for _ in range(11)]
    new = [rng.randint(0, top) for _ in hist]
    new[3] = top
    x = batch8(heads, kv, dim, 16 if top == 4 else 64, hist, new, seed=top, pad_rows=1)
    out, b = run8(x)
    b.check()
    check_rows(x, out)


@pytest.mark.parametrize("heads,kv,dim", HEADS)
@pytest.mark.parametrize("page", [16, 64, 128])
def test_many_new_tokens(heads, kv, dim, page):
    hist = [0, 0, 130, 1000, 513, 77, 0]
    new = [1, 300, 257, 1, 128, 0, 43]
    x = batch8(heads, kv, dim, page, hist, new, seed=page, pad_rows=2, packed=page == 16)
    out, b = run8(x)
    b.check()
    check_rows(x, out)


@pytest.mark.parametrize("window", [1, 50, 64, 700])
@pytest.mark.parametrize("top", [1, 5, 200])
def test_window(window, top):
    """The last W slots only: pages wholly before every row's window may be gone (their
    table entries are junk) and slots there hold NaN."""
    rng = random.Random(window)
    hist = [0, 10, 49, 50, 63, 64, 200, 900]
    new = [rng.randint(1, top) for _ in hist]
    x = Batch(12, 2, 128, 16, hist, new, seed=window)
    keep = x.table.clone()
    for i, h in enumerate(hist):
        gone = max(0, h + 1 - window) // 16
        for pg in keep[i, :gone].tolist():
            x.k_pages[pg] = float("nan")
            x.v_pages[pg] = float("nan")
        x.table[i, :gone] = 10 ** 8
    x = in_8_bits(x)
    out, b = run8(x, window)
    b.check()
    x.table = keep
    check_rows(x, out, window)


def prefix_launches8(b, run):
    before = b.timing_table().get("attn_paged_prefix_kv8", (0, 0))[1]
    b.timing(True)
    out = run()
    b.timing_collect()
    b.timing(False)
    return out, b.timing_table().get("attn_paged_prefix_kv8", (0, 0))[1] - before


def shared_prefix(heads, kv, dim, prefix, page, top, seqs):
    rng = random.Random(prefix + top)
    hist = [prefix + (0, 1, 17, 64, 100, 300, 0)[i % 7] for i in range(seqs)]
    new = [rng.randint(1, top) for _ in hist]
    new[4] = 0
    x = batch8(heads, kv, dim, page, hist, new, seed=top, prefix=prefix, pad_rows=2)
    keep = x.table.clone()
    x.table[:, :prefix // page] = -3
    out, b = run8(x, max_new=top)
    b.check()
    x.table = keep
    check_rows(x, out)


@pytest.mark.parametrize("heads,kv,dim", HEADS)
@pytest.mark.parametrize("prefix,page", [(16, 16), (128, 64), (1040, 16)])
@pytest.mark.parametrize("top", [1, 3, 150])
def test_short_shared_prefix(heads, kv, dim, prefix, page, top):
    shared_prefix(heads, kv, dim, prefix, page, top, 7)


@pytest.mark.parametrize("heads,kv,dim,prefix,page,top,seqs", [
    (12, 2, 128, 1040, 16, 1, 130), (12, 2, 128, 4096, 64, 4, 40), (12, 2, 128, 7056, 16, 30, 70),
    (32, 2, 128, 2064, 16, 1, 70), (32, 2, 128, 9600, 128, 2, 30), (4, 2, 64, 2048, 32, 1, 100),
    (16, 16, 64, 2064, 16, 1, 16), (16, 16, 64, 2048, 128, 9, 16), (16, 16, 64, 3088, 16, 40, 20),
    (8, 4, 128, 2080, 32, 1, 60), (32, 8, 64, 2064, 16, 5, 30), (16, 2, 64, 4128, 32, 1, 40)])
def test_long_shared_prefix(heads, kv, dim, prefix, page, top, seqs):
    shared_prefix(heads, kv, dim, prefix, page, top, seqs)


@pytest.mark.parametrize("hist,new", [([20000], [1]), ([9000, 3], [1, 4]), ([5000], [700])])
def test_one_long_sequence_is_cut_over_the_gpu(hist, new):
    x = batch8(12, 2, 128, 64, hist, new, seed=1)
    out, b = run8(x)
    b.check()
    check_rows(x, out)


def test_many_short_sequences():
    rng = random.Random(5)
    x = batch8(4, 2, 64, 16, [rng.randint(0, 70) for _ in range(1500)], [1] * 1500, seed=5)
    out, b = run8(x)
    b.check()
    check_rows(x, out)


@pytest.mark.parametrize("heads,kv,dim,top", [(16, 1, 64, 2), (12, 2, 128, 2), (8, 4, 128, 1),
                                              (12, 2, 128, 5), (4, 2, 64, 1)])
def test_short_pieces_one_after_another_give_the_same_bits(heads, kv, dim, top):
    """Every tile ends a piece: a warp is in the next piece while another still finishes the
    one before."""
    rng = random.Random(21)
    hist = [rng.randint(0, 62) for _ in range(2000)]
    x = batch8(heads, kv, dim, 32, hist, [rng.randint(1, top) for _ in hist], seed=21)
    first, b = run8(x)
    b.check()
    check_rows(x, first)
    for _ in range(20):
        out, _ = run8(x)
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("heads,kv,dim,top", [(12, 2, 128, 1), (12, 2, 128, 2), (12, 2, 128, 4),
                                              (4, 2, 64, 1), (32, 8, 64, 3), (16, 1, 64, 2)])
@pytest.mark.parametrize("prefix", [0, 8192])
def test_pieces_of_which_most_warps_see_nothing(heads, kv, dim, top, prefix):
    """Sequences of a few slots and of some hundred in turn, cut and whole: warps that find
    nothing in a piece are far ahead in the next while the others end it."""
    hist = [prefix + 3, prefix + 500] * 45
    x = batch8(heads, kv, dim, 64, hist, [top] * 90, seed=25, prefix=prefix)
    first, b = run8(x)
    b.check()
    check_rows(x, first)
    for _ in range(10):
        out, _ = run8(x)
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("top", [1, 5, 60])
def test_a_workspace_keeps_nothing_of_the_call_before(top):
    b = block(12, 2, 128)
    ws = torch.zeros(b.attn_paged_workspace_bytes(2000, 400), dtype=torch.uint8, device="cuda")
    for seed, (hist, new) in enumerate([
            ([6000] * 6, [top] * 6), ([6000] * 6, [0, top, 0, 0, 1, 0]),
            ([3] * 152, [1] * 152), ([700] * 153, [0, 1, 1] * 51), ([9000, 2, 4000], [1, top, 0]),
            ([9000], [top]), ([0] * 6, [0] * 5 + [1]), ([800] * 4, [1, 1, top, 1])]):
        x = batch8(12, 2, 128, 64, hist, new, seed=30 + seed, pad_rows=1)
        bad = [1] if len(hist) == 4 else []
        d = x.descriptor(b, max_new=max(new + [1]))
        if bad:
            x.lens[1] = -1
        out = torch.full((x.rows, 12, 128), MARK, dtype=torch.float16, device="cuda")
        b.attn_paged_kv8(d, x.q, *x.pools8, out, ws)
        if bad:
            with pytest.raises(blk.BlkError):
                b.check()
        else:
            b.check()
        check_rows(x, out, skip=bad)


@pytest.mark.parametrize("top", [1, 4, 40])
@pytest.mark.parametrize("prefix", [0, 8192])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_stays_nan_and_alone(top, prefix, value):
    hist = [prefix + h for h in (3, 9000, 500)] * (1 if prefix == 0 else 30)
    x = batch8(12, 2, 128, 64, hist, [top, 1, top] * (len(hist) // 3), seed=22, prefix=prefix)
    want, bound = x.reference()
    x.q[0, 3] = value
    x.q[top, 7] = value
    x.q[2 * top, 11] = value
    out, b = run8(x)
    b.check()
    off, bad = (out.double() - want).abs() <= bound, torch.zeros(x.rows, 12, dtype=torch.bool)
    bad[0, 3] = bad[top, 7] = bad[2 * top, 11] = True
    assert out[bad].isnan().all() and off[~bad].all()


@pytest.mark.parametrize("top", [1, 5, 60])
def test_a_visible_block_of_nan_reaches_its_rows_and_no_other_sequence(top):
    """A NaN among a visible key's values makes its sequence's rows of that kv head NaN (the
    rows before it may be too); one among the values its columns' block."""
    x = Batch(12, 2, 128, 64, [200, 100, 300], [top, 1, top], seed=23)
    x.k_pages[int(x.table[0, 1]), 1, 5, 70] = float("nan")
    x.v_pages[int(x.table[2, 0]), 0, 9, 33] = float("inf")
    x = in_8_bits(x)
    out, b = run8(x)
    b.check()
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[:top, 6:] = True
    bad[top + 1:, :6, 32:64] = True
    assert out[bad].isnan().all()
    for pool in (x.k_pages, x.v_pages):          # all else is as without those blocks
        pool.nan_to_num_(0.0)
    want, bound = x.reference()
    assert ((out.double() - want).abs() <= bound)[~bad].all()


@pytest.mark.parametrize("top", [1, 100])
def test_scores_of_any_size(top):
    x = batch8(12, 2, 128, 64, [700, 64], [top, 1], seed=6)
    x.q[0] *= 40.0
    x.q[-1] *= 0.0
    out, b = run8(x)
    b.check()
    want, _ = x.reference()
    got = out.double()
    assert torch.isfinite(got).all()
    # scores of 40 times the size have 40 times the absolute error (2^-13 * 40 of A);
    # an all-zero q is the mean of V
    v_max = 6.0
    assert ((got[0] - want[0]).abs() <= (2.0 ** -10 + 40 * 2.0 ** -13) * v_max).all()
    assert ((got[-1] - want[-1]).abs() <= 2.0 ** -10 * v_max).all()


@pytest.mark.parametrize("top", [1, 5, 60])
@pytest.mark.parametrize("k_gain,v_gain", [(1e-4, 1e-6), (1.0, 9000.0), (2e-7, 1.0), (1e-3, 60000.0 / 6)])
def test_pools_of_any_magnitude(top, k_gain, v_gain):
    """Values from fp16's least to its greatest: scales of E5M2's subnormals and of 2^15.
    (The queries bring the scores back to the size that the bound is for.)"""
    x = Batch(12, 2, 128, 64, [300, 70, 1000], [top, 1, top], seed=24)
    x.k_pages *= k_gain
    x.v_pages.copy_((x.v_pages.double() * v_gain).clamp(-65504, 65504))
    x.q *= min(1 / k_gain, 10000.0)
    x = in_8_bits(x)
    out, b = run8(x)
    b.check()
    check_rows(x, out)


def test_offsets_past_32_bits():
    """Pools of 2^32 codes and more: pages at their end."""
    n_pages = (1 << 32) // (2 * 128 * 128) + 5
    x = batch8(12, 2, 128, 128, [300, 4000], [1, 1], seed=7, n_pages=n_pages, junk=0.0)
    for pool in (x.k_pages, x.v_pages, *(t.view(torch.uint8) for t in x.pools8)):
        pool[n_pages - 2] = pool[int(x.table[0, 1])]
    x.table[0, 0] = n_pages - 2
    out, b = run8(x)
    b.check()
    check_rows(x, out)
    # and the append and the read there
    slots = torch.tensor([(n_pages - 1) * 128 + 127, (n_pages - 3) * 128], device="cuda")
    k = torch.randn((2, 2, 128), device="cuda").half()
    back = [torch.empty_like(k) for _ in range(2)]
    b.page_append_kv8(k, -k, slots, *x.pools8)
    b.page_read_kv8(slots, *x.pools8, *back)
    b.check()
    want = values(*quantise(k))
    assert torch.equal(back[0].double(), want) and torch.equal(back[1].double(), -want)
    assert torch.equal(x.pools8[0][n_pages - 1, :, 127], quantise(k)[0][0])


@pytest.mark.parametrize("top", [1, 90])
def test_refused_sequences_leave_their_rows_and_the_others_are_served(top):
    new = [1, top, 1, 2]
    x = batch8(12, 2, 128, 16, [30, 40, 500, 60], new, seed=8)
    out, b = run8(x, max_len=40 + top)
    with pytest.raises(blk.BlkError) as e:
        b.check()
    assert e.value.status == blk.BLK_ERR_PAGE
    check_rows(x, out, skip=[i for i, h in enumerate(x.hist) if h + new[i] > 40 + top])
    b.check()                                    # reported once
    x.lens[2] = -4
    out, b = run8(x)
    with pytest.raises(blk.BlkError):
        b.check()
    check_rows(x, out, skip=[2])
    for prefix, seqs in ((64, 3), (4096, 60)):
        x = batch8(12, 2, 128, 64, [prefix, prefix + 1, prefix] * (seqs // 3),
                   [1, top if seqs < 9 else 3, 1] * (seqs // 3), seed=9, prefix=prefix)
        short = [i for i in (0, 7, 8, 9, 31, 59) if i < seqs]
        for i in short:
            x.lens[i] = prefix - 1
        out, b = run8(x)
        with pytest.raises(blk.BlkError):
            b.check()
        check_rows(x, out, skip=short)


@pytest.mark.parametrize("top", [1, 60])
@pytest.mark.parametrize("bad", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
def test_a_bad_page_reads_as_zeros_and_is_reported(top, bad):
    x = batch8(12, 2, 128, 16, [100, 40], [top, 1], seed=10)
    pg = int(x.table[0, 2])
    x.table[0, 2] = bad
    out, b = run8(x)
    with pytest.raises(blk.BlkError) as e:
        b.check()
    assert e.value.status == blk.BLK_ERR_PAGE
    x.table[0, 2] = pg
    x.k_pages[pg] = 0
    x.v_pages[pg] = 0
    check_rows(x, out)


@pytest.mark.parametrize("top", [1, 4, 40])
@pytest.mark.parametrize("prefix", [0, 128, 32768])
def test_a_captured_graph_serves_other_lengths(top, prefix):
    """Lengths, row ranges, tables, codes and scales are the device's: a graph captured at one
    step replays the next, with the same bits as the call itself."""
    x = batch8(12, 2, 128, 64, [prefix + h for h in (100, 7, 300)], [top, 1, 2], seed=11,
               prefix=prefix)
    y = batch8(12, 2, 128, 64, [prefix + h for h in (220, 64, 1)], [1, 2, top], seed=12,
               prefix=prefix)
    b = block(12, 2, 128)
    n_pages = max(x.k_pages.shape[0], y.k_pages.shape[0])
    rows, blocks = max(x.rows, y.rows), max(x.max_blocks, y.max_blocks)
    pools = [torch.zeros((n_pages, *t.shape[1:]), dtype=torch.uint8, device="cuda").view(t.dtype)
             for t in x.pools8]
    q = torch.zeros((rows, 12, 128), dtype=torch.float16, device="cuda")
    table = torch.full((3, blocks), -1, dtype=torch.int32, device="cuda")
    lens, start = torch.zeros_like(x.lens), torch.zeros_like(x.row_start)
    pre = torch.zeros(prefix // 64, dtype=torch.int32, device="cuda") if prefix else None
    out = torch.full((rows, 12, 128), MARK, dtype=torch.float16, device="cuda")
    ws = torch.empty(b.attn_paged_workspace_bytes(rows, 3), dtype=torch.uint8, device="cuda")
    d = b.paged_batch(start, lens, table, rows, 64, n_pages, max(2, top), blocks * 64,
                      prefix_pages=pre)

    def load(z):
        for to, src in zip(pools, z.pools8):
            to.view(torch.uint8)[:src.shape[0]] = src.view(torch.uint8)
        q[:z.rows] = z.q
        table.fill_(-1)
        table[:, :z.max_blocks] = z.table
        lens.copy_(z.lens)
        start.copy_(z.row_start)
        if prefix:
            pre.copy_(z.prefix)
        out.fill_(MARK)

    load(x)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            b.attn_paged_kv8(d, q, *pools, out, ws, stream=s)
    for z in (x, y, x):
        load(z)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        b.check()
        check_rows(z, out)
        again = torch.full_like(out, MARK)
        b.attn_paged_kv8(d, q, *pools, again, ws)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def test_two_streams_with_their_own_workspaces():
    xs = [batch8(12, 2, 128, 64, [2000 + 31 * i, 5, 700], [1, 1 + i % 3, 60 * (i % 2)], seed=20 + i)
          for i in range(4)]
    streams, args = [torch.cuda.Stream() for _ in xs], []
    b = block(12, 2, 128)
    for x in xs:
        out = torch.full((x.rows, 12, 128), MARK, dtype=torch.float16, device="cuda")
        ws = torch.empty(b.attn_paged_workspace_bytes(x.rows, 3), dtype=torch.uint8, device="cuda")
        args.append((x.descriptor(b), out, ws))
    torch.cuda.synchronize()
    for _ in range(5):
        for x, (d, out, ws), s in zip(xs, args, streams):
            b.attn_paged_kv8(d, x.q, *x.pools8, out, ws, stream=s)
    torch.cuda.synchronize()
    b.check()
    for x, (_, out, _) in zip(xs, args):
        check_rows(x, out)


@pytest.mark.parametrize("top", [2, 90])
@pytest.mark.parametrize("first,width", [(32, 64), (8, 24), (0, 8)])
def test_strided_output_and_the_gaps_between_rows(top, first, width):
    x = batch8(12, 2, 128, 64, [70, 200], [2, top], seed=13)
    wide = torch.full((x.rows, 12 * 128 + width), MARK, dtype=torch.float16, device="cuda")
    out, b = run8(x, out=wide[:, first:first + 12 * 128].unflatten(1, (12, 128)))
    b.check()
    check_rows(x, out)
    assert (wide[:, :first] == MARK).all() and (wide[:, first + 12 * 128:] == MARK).all()


@pytest.mark.parametrize("new,prefix", [([1, 3, 1], 0), ([60, 3, 90], 0), ([1, 3, 1] * 40, 4096)])
def test_a_workspace_at_a_16_byte_boundary(new, prefix):
    x = batch8(12, 2, 128, 64, [prefix + h for h in (900, 4000, 0)] * (len(new) // 3), new, seed=15,
               prefix=prefix)
    out, b = run8(x, shift=16)
    b.check()
    check_rows(x, out)


@pytest.mark.parametrize("top", [1, 5, 70])
def test_rows_before_the_first_sequence_and_idle_batches(top):
    x = batch8(12, 2, 128, 64, [100, 7], [1, top], seed=16, pad_rows=4)
    x.row_start += 3
    x.q[3:3 + x.n] = x.q[:x.n].clone()
    out, b = run8(x)
    b.check()
    assert (out[:3] == MARK).all()
    x.q = x.q[3:]
    x.rows -= 3
    check_rows(x, out[3:])
    for prefix in (0, 8192):
        x = batch8(12, 2, 128, 64, [prefix + 5] * 80, [0] * 80, seed=17, prefix=prefix, pad_rows=top)
        out, b = run8(x, max_new=top)
        b.check()
        assert (out == MARK).all()


@pytest.mark.parametrize("top", [2, 50])
def test_more_new_tokens_than_announced_are_refused(top):
    x = batch8(12, 2, 128, 64, [100, 7, 30], [1, top, 1], seed=18)
    out, b = run8(x, max_new=top - 1)
    with pytest.raises(blk.BlkError) as e:
        b.check()
    assert e.value.status == blk.BLK_ERR_PAGE
    check_rows(x, out, skip=[1])
    x.row_start[1] = x.rows + 5                  # row ranges that run backwards or past the batch
    out, b = run8(x)
    with pytest.raises(blk.BlkError):
        b.check()
    assert (out[:1 + top] == MARK).all()


@pytest.mark.parametrize("nats", [9.0, 15.0, 17.4])
@pytest.mark.parametrize("at", [0, 70, 8000])
@pytest.mark.parametrize("heads,kv,dim,top", [(12, 2, 128, 1), (12, 2, 128, 5), (4, 2, 64, 2),
                                              (12, 2, 128, 50), (16, 16, 64, 40)])
def test_small_weights(heads, kv, dim, top, at, nats):
    """One slot outweighs all others by up to e^17 and hides nothing of them."""
    x = Batch(heads, kv, dim, 64, [32000, 90, 9000, 4], [1, top, top, 1], seed=41)
    x = in_8_bits(with_sink(x, at, nats))
    out, b = run8(x)
    b.check()
    check_weights(x, out, K8_FEW if top * heads // kv <= 32 else K_MANY)


@pytest.mark.parametrize("top", [1, 60])
@pytest.mark.parametrize("prefix", [0, 8192])
def test_a_slot_far_above_all_others_is_the_result(top, prefix):
    """Scores of 10^7 and more, whose fp32 values are whole numbers apart: weights stay in
    fp16's range, and the row is that slot's V (its weight and the result rounded once each)."""
    hist = [prefix + 200 + 37 * (i % 5) for i in range(60)]
    x = Batch(12, 2, 128, 64, hist, [top] + [1] * 59, seed=44, prefix=prefix)
    x.k_pages[~x.k_pages.isnan()] = 0
    x.q[..., 0] = 30000
    where, r0 = [], 0
    for b, (have, more) in enumerate(zip(x.hist, x.new)):
        for g in range(2):
            at = prefix + 3 * b + g
            pg = int(x.table[b, at // 64])
            x.k_pages[pg, g, at % 64, 0] = 8000 + 199 * b + 64 * g
            where.append((r0, more, g, pg, at % 64))
        r0 += more
    x = in_8_bits(x)
    want = torch.empty_like(x.q)
    for r0, more, g, pg, s in where:
        want[r0:r0 + more, g * 6:g * 6 + 6] = x.v_pages[pg, g, s]
    out, b = run8(x)
    b.check()
    off = (out.double() - want.double()).abs()
    assert (off <= (2 * U16 + 2.0 ** -13) * want.double().abs() + 2.0 ** -25).all()


@pytest.mark.parametrize("step", [60, 200, -94])
@pytest.mark.parametrize("k0", [12000, 25000])
@pytest.mark.parametrize("top,prefix", [(1, 0), (5, 0), (60, 0), (1, 8192)])
def test_large_scores_that_rise_from_tile_to_tile(top, prefix, k0, step):
    """Scores of 3 - 7 10^7 that grow or fall from one 128 slots to the next: a row stays
    between the least and the greatest of V (see the fp16 caches' test)."""
    hist = [prefix + 900 + 37 * (i % 5) for i in range(60)]
    x = Batch(12, 2, 128, 128, hist, [top] + [1] * 59, seed=45, prefix=prefix)
    seen = ~x.k_pages.isnan()
    x.k_pages[seen] = 0
    x.v_pages[seen] = 1 + x.v_pages[seen].abs().clamp(max=1)
    x.q[..., 0], x.q[..., 40] = 30000, 1
    for b, (have, more) in enumerate(zip(x.hist, x.new)):
        for j in range(-(-(have + more) // 128)):
            pg = int(x.table[b, j])
            x.k_pages[pg, :, :, 0] = torch.where(seen[pg, :, :, 0], k0, x.k_pages[pg, :, :, 0])
            x.k_pages[pg, :, :, 40] = torch.where(seen[pg, :, :, 40], 94 * 100 + step * (j - 60),
                                                  x.k_pages[pg, :, :, 40])
    x = in_8_bits(x)
    lo, hi = x.v_pages[seen].min().item(), x.v_pages[seen].max().item()
    out, b = run8(x)
    b.check()
    got = out[:x.n].double()
    assert got.min().item() >= lo * (1 - 2 * U16 - 2.0 ** -13)
    assert got.max().item() <= hi * (1 + 2 * U16 + 2.0 ** -13)


def test_equals_the_fp16_cache_that_holds_the_same_values():
    """Within both results' bounds of one another, few rows and many."""
    from test_paged_gpu import run_attention
    for top in (1, 4, 70):
        x = batch8(12, 2, 128, 64, [500, 0, 1300], [top, 1, 2], seed=47)
        a, b = run8(x)
        c, _ = run_attention(x)
        b.check()
        _, bound = x.reference()
        assert ((a.double() - c.double()).abs()[:x.n] <= 2 * bound[:x.n]).all()


def test_argument_errors():
    x = batch8(12, 2, 128, 64, [70, 200], [1, 2], seed=14, prefix=64)
    b = block(12, 2, 128)
    nb = b.attn_paged_workspace_bytes(x.rows, 2)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    out = torch.full((x.rows, 12, 128), MARK, dtype=torch.float16, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    P = [t.data_ptr() for t in x.pools8]

    def call(expect, handle=b.handle, q=x.q.data_ptr(), q_stride=1536, o_stride=1536,
             ws_bytes=nb, pool=P, **kw):
        d = x.descriptor(b)
        for name, val in kw.items():
            setattr(d, name, val)
        rc = blk.blk_attn_paged_kv8(handle, d, q, q_stride, blk.BlkKv8Pool(*pool) if pool else None,
                                    out.data_ptr(), o_stride, ws.data_ptr(), ws_bytes, st)
        assert rc == expect, (rc, kw)

    S, A, N = blk.BLK_ERR_SHAPE, blk.BLK_ERR_ALIGN, blk.BLK_ERR_NULL
    call(N, handle=None)
    call(N, q=None)
    call(N, pool=None)
    for i in range(4):
        call(N, pool=[*P[:i], None, *P[i + 1:]])
        call(A, pool=[*P[:i], P[i] + 8, *P[i + 1:]])
    call(N, row_start=None)
    call(N, prefix_pages=None)
    call(A, q=x.q.data_ptr() + 2)
    call(A, q_stride=1540)
    call(S, q_stride=1528)
    call(S, o_stride=0)
    call(S, page_size=48)
    call(S, n_pages=0)
    call(S, n_seqs=4097)
    call(S, n_rows=0)
    call(S, max_new=0)
    call(S, max_len=0)
    call(S, prefix_len=65)
    call(blk.BLK_ERR_CACHE_OVERFLOW, max_len=x.max_blocks * 64 + 1)
    call(blk.BLK_ERR_WORKSPACE, ws_bytes=nb - 1)
    call(S, handle=block(12, 2, 128, 50).handle)        # a prefix and a window
    torch.cuda.synchronize()
    assert (out == MARK).all()
    d = x.descriptor(b)
    p = x.pools8
    for bad in (dict(q=x.q[:1]), dict(q=x.q.float()), dict(out=out.cpu()),
                *(dict(pool=[t[:-1] if i == j else t for j, t in enumerate(p)]) for i in range(4)),
                *(dict(pool=[t.view(torch.int8) if i == j else t for j, t in enumerate(p)])
                  for i in range(4))):
        with pytest.raises(blk.BlkError) as e:
            b.attn_paged_kv8(d, bad.get("q", x.q), *bad.get("pool", p), bad.get("out", out), ws)
        assert e.value.status == S
    with pytest.raises(blk.BlkError) as e:
        b.attn_paged_kv8(d, x.q, *p, out, ws.cpu())
    assert e.value.status == blk.BLK_ERR_WORKSPACE
    assert NAN_SCALE == 0x7f


@pytest.mark.parametrize("heads,kv,dim,top", [(12, 2, 128, 1), (12, 2, 128, 2), (12, 2, 128, 4),
                                              (8, 2, 128, 8), (8, 8, 64, 7), (16, 4, 64, 3),
                                              (16, 4, 64, 6), (16, 4, 64, 8), (16, 4, 64, 30)])
@pytest.mark.parametrize("k_gain,v_gain", [(9000.0, 9000.0), (9000.0, 1e-6), (1e-4, 9000.0)])
def test_large_scales_at_every_number_of_rows(heads, kv, dim, top, k_gain, v_gain):
    """Scales above 3584 in K, in V and in both, for 1 - 4 tiles of rows and for many."""
    x = Batch(heads, kv, dim, 64, [300, 70, 1000], [top, 1, top], seed=48)
    for pool, gain in ((x.k_pages, k_gain), (x.v_pages, v_gain)):
        pool.copy_((pool.double() * gain).clamp(-65504, 65504))
    x.q.copy_(x.q.double() / k_gain)         # (the scores' size is the one that the bound is for)
    x = in_8_bits(x)
    out, b = run8(x)
    b.check()
    check_rows(x, out)


@pytest.mark.parametrize("heads,kv,dim,top", [(12, 2, 128, 2), (12, 2, 128, 4), (16, 4, 64, 3),
                                              (16, 4, 64, 6), (16, 4, 64, 8)])
def test_rows_of_large_and_small_scores_beside_one_another(heads, kv, dim, top):
    """Heads whose scores pass 2^22 in the same tiles of rows as heads whose scores do not: the
    former take the V of the slot that is far above all others, the latter keep to their bound."""
    x = Batch(heads, kv, dim, 64, [500, 90, 1200], [top, 1, top], seed=49)
    x.k_pages[..., 0].copy_(torch.where(x.k_pages[..., 0].isnan(), x.k_pages[..., 0], 0))
    big = torch.arange(heads, device="cuda") % 3 == 1
    at = [(0, 1, 5), (1, 0, 60), (2, 10, 17)]           # (sequence, page of its table, slot of it)
    x.q[..., 0] = 0
    for b_, blk_, s in at:
        x.k_pages[int(x.table[b_, blk_]), :, s, :] = 0
        x.k_pages[int(x.table[b_, blk_]), :, s, 0] = 16000
    x = in_8_bits(x)
    want, bound = x.reference()
    x.q[:, big, 0] = 30000
    out, b = run8(x)
    b.check()
    off = (out.double() - want).abs()
    assert (off <= bound)[:, ~big].all()
    r0 = 0
    for (b_, blk_, s), n in zip(at, x.new):
        v = x.v_pages[int(x.table[b_, blk_]), :, s].double().repeat_interleave(heads // kv, 0)[big]
        got = out[r0:r0 + n, big].double()
        assert ((got - v).abs() <= (2 * U16 + 2.0 ** -13) * v.abs() + 2.0 ** -25).all()
        r0 += n
