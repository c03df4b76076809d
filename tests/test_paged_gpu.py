"""GPU tests of the paged cache's operators: the plan against the same sums on the
host, the append bit for bit, the attention against a 64-bit evaluation of its
definition within the bound that its roundings give (tests/paged_reference.py)."""
import random
from types import SimpleNamespace

import pytest
import torch

import decode_qwen2_block_gb300 as blk
from paged_reference import Batch

pytestmark = pytest.mark.gpu
MARK = -77.0           # what an output holds where nothing may be written
_blocks = {}


def block(heads, kv, dim, window=0):
    key = (heads, kv, dim, window)
    if key not in _blocks:
        s = SimpleNamespace(hidden=heads * dim, n_heads=heads, n_kv_heads=kv, head_dim=dim,
                            intermediate=heads * dim, has_qkv_bias=False, rms_eps=1e-6,
                            rope_theta=1e4)
        _blocks[key] = blk.Block(s, 256)
        _blocks[key].set_window(window)
    return _blocks[key]


# ---------------------------------------------------------------------- plan
def host_plan(page, lens, news, free, table, n_rows):
    """The plan of blk.h on the host; (table, starts, slots, pos, used, refused)."""
    table = [list(r) for r in table]
    cap = len(table[0]) * page
    starts, slots, pos, used, take, refused = [0], [-1] * n_rows, [0] * n_rows, 0, 0, []
    for b, (have, more) in enumerate(zip(lens, news)):
        r0 = starts[-1]
        rows = more if 0 <= more <= n_rows else 0
        starts.append(r0 + rows)
        ok = 0 <= more <= n_rows and r0 + rows <= n_rows and 0 <= have <= cap and have + more <= cap
        if ok:
            held, need = -(-have // page), -(-(have + more) // page) - -(-have // page)
            ok = need == 0 or take + need <= len(free)
            if ok:
                for i in range(need):
                    table[b][held + i] = free[take + i]
                used = max(used, take + need) if need else used
            take += need
        if not ok:
            refused.append(b)
            continue
        for t in range(more):
            p = have + t
            pg = table[b][p // page]
            slots[r0 + t] = -1 if pg < 0 else pg * page + p % page
            pos[r0 + t] = p
    return table, starts, slots, pos, used, refused


def run_plan(page, lens, news, n_free, n_rows, max_blocks, seed=0, check=True):
    rng = random.Random(seed)
    B = len(lens)
    ids = list(range(10 ** 6, 10 ** 6 + n_free))
    rng.shuffle(ids)
    table = [[rng.randrange(1000) if i < -(-max(0, n) // page) else -5 for i in range(max_blocks)]
             for n in lens]
    want = host_plan(page, lens, [1] * B if news is None else news, ids, table, n_rows)
    i64 = dict(dtype=torch.int64, device="cuda")
    tab = torch.tensor(table, dtype=torch.int32, device="cuda")
    free = torch.tensor(ids, dtype=torch.int32, device="cuda")
    start, slots = torch.full((B + 1,), -9, **i64), torch.full((n_rows,), -9, **i64)
    pos, used = torch.full((n_rows,), -9, **i64), torch.full((1,), -9, **i64)
    b = block(4, 2, 64)
    b.page_plan(page, torch.tensor(lens, **i64), None if news is None else torch.tensor(news, **i64),
                free, tab, start, slots, pos, used)
    got = (tab.tolist(), start.tolist(), slots.tolist(), pos.tolist(), used.item())
    for name, g, w in zip(("table", "row_start", "slot_map", "pos", "used"), got, want):
        assert g == w, name
    if want[5]:
        with pytest.raises(blk.BlkError) as e:
            b.check()
        assert e.value.status == blk.BLK_ERR_PAGE
    else:
        b.check()
    return want


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("B,hi,new_hi", [(1, 0, 1), (5, 300, 40), (513, 90, 7), (4096, 33, 2)])
def test_plan(page, B, hi, new_hi):
    rng = random.Random(B + page)
    lens = [rng.randint(0, hi) for _ in range(B)]
    news = [rng.randint(0, new_hi) for _ in range(B)]
    news[0] = max(1, news[0])
    want = run_plan(page, lens, news, sum(news) + 3, sum(news) + 5, -(-(hi + new_hi) // page) + 1)
    assert not want[5]


def test_plan_one_token_each_without_new_lens():
    run_plan(64, [0, 63, 64, 65, 127, 128], None, 4, 6, 3)


def test_plan_one_long_prompt_fills_many_ctas():
    run_plan(16, [3, 0, 9], [0, 100003, 1], 6300, 100004, 6300)


def test_plan_refuses_what_does_not_fit_and_serves_the_rest():
    # too few free pages for sequence 2; 3 needs none; 4 comes after the list ran out
    want = run_plan(16, [0, 5, 16, 30, 16], [20, 3, 40, 2, 1], 3, 66, 8)
    assert want[5] == [2, 4]
    # a negative and an overlong length, a negative and a huge number of tokens
    want = run_plan(16, [-1, 4, 200, 7, 7, 0], [2, 2, 1, -3, 10 ** 15, 2], 8, 32, 8)
    assert want[5] == [0, 2, 3, 4]
    # rows that do not fit the row arrays
    want = run_plan(32, [0, 0, 0], [10, 10, 10], 8, 25, 4)
    assert want[5] == [2]


# -------------------------------------------------------------------- append
@pytest.mark.parametrize("kv,dim,page", [(2, 128, 64), (8, 64, 16), (1, 128, 128), (2, 64, 32)])
@pytest.mark.parametrize("n", [1, 77, 5000])
@pytest.mark.parametrize("layout", ["rows", "packed", "heads"])
def test_append(kv, dim, page, n, layout):
    gen = torch.Generator("cuda")
    gen.manual_seed(n)
    n_pages = -(-n // page) + 2
    if layout == "rows":
        k, v = (torch.randn((n, kv, dim), generator=gen, device="cuda").half() for _ in range(2))
    elif layout == "packed":     # slices of a fused projection's rows
        x = torch.randn((n, 6 * kv * dim), generator=gen, device="cuda").half()
        k, v = (x[:, i * kv * dim:(i + 1) * kv * dim].unflatten(1, (kv, dim)) for i in (4, 5))
    else:                        # slots of a contiguous cache
        c = torch.randn((2, kv, n + 9, dim), generator=gen, device="cuda").half()
        k, v = c[0, :, 4:4 + n].transpose(0, 1), c[1, :, 4:4 + n].transpose(0, 1)
    slots = torch.randperm(n_pages * page, generator=gen, device="cuda")[:n]
    if n > 3:
        slots[n // 2] = -1
    pools = [torch.full((n_pages, kv, page, dim), MARK, dtype=torch.float16, device="cuda")
             for _ in range(2)]
    b = block(kv * 2, kv, dim)
    b.page_append(k, v, slots, *pools)
    b.check()
    for pool, rows in zip(pools, (k, v)):
        want = torch.full((n_pages * page, kv, dim), MARK, dtype=torch.float16, device="cuda")
        keep = slots >= 0
        want[slots[keep]] = rows[keep]
        got = pool.transpose(1, 2).reshape(-1, kv, dim)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_append_reports_a_slot_outside_the_pool_and_writes_nothing_there():
    k = torch.ones((3, 2, 64), dtype=torch.float16, device="cuda")
    pools = [torch.zeros((4, 2, 16, 64), dtype=torch.float16, device="cuda") for _ in range(2)]
    b = block(4, 2, 64)
    b.page_append(k, k, torch.tensor([64, 5, -2], device="cuda"), *pools)
    with pytest.raises(blk.BlkError) as e:
        b.check()
    assert e.value.status == blk.BLK_ERR_PAGE
    for pool in pools:
        assert pool.sum().item() == 2 * 64 and (pool[0, :, 5] == 1).all()


# ----------------------------------------------------------------- attention
def run_attention(x, window=0, out=None, stream=None, shift=0, **kw):
    b = block(x.heads, x.kv, x.dim, window)
    d = x.descriptor(b, **kw)
    if out is None:
        out = torch.full((x.rows, x.heads, x.dim), MARK, dtype=torch.float16, device="cuda")
    nb = b.attn_paged_workspace_bytes(x.rows, len(x.hist), prefix=d.prefix_len > 0)
    ws = torch.full((nb + 32,), 255, dtype=torch.uint8, device="cuda")     # NaN wherever it is read
    ws = ws[shift:shift + nb]
    b.attn_paged(d, x.q, x.k_pages, x.v_pages, out, ws, stream=stream)
    return out, b


def check_rows(x, out, window=0, skip=()):
    want, bound = x.reference(window, skip)
    at = 0
    for i, t in enumerate(x.new):
        got = out[at:at + t].double()
        if i in skip:
            assert (got == MARK).all(), f"sequence {i} is refused: its rows stay"
        elif t:
            off = (got - want[at:at + t]).abs()
            worst = (off / bound[at:at + t]).max().item()
            assert torch.isfinite(got).all() and worst <= 1.0, f"sequence {i}: {worst:.3g} of the bound"
        at += t
    assert (out[at:] == MARK).all(), "rows behind the batch stay"


HEADS = [(12, 2, 128), (32, 2, 128), (4, 2, 64), (16, 16, 64), (8, 4, 128), (32, 8, 64), (16, 2, 64),
         (4, 4, 128), (16, 1, 64)]


@pytest.mark.parametrize("heads,kv,dim", HEADS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_decode(heads, kv, dim, page):
    """One token per sequence, histories from none to many tiles, an idle sequence, junk
    (NaN) in every slot past a sequence's last and in every other page."""
    hist = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 1000, 0, 300]
    new = [1] * len(hist)
    new[-1] = 0
    x = Batch(heads, kv, dim, page, hist, new, seed=page + heads, pad_rows=3, packed=page == 32)
    out, b = run_attention(x)
    b.check()
    check_rows(x, out)


@pytest.mark.parametrize("heads,kv,dim", HEADS)
@pytest.mark.parametrize("top", [2, 4, 9])
def test_few_new_tokens(heads, kv, dim, top):
    """Drafts to verify: up to nine tokens per sequence (the few-row kernel in each of
    its row counts, or the many-row kernel for large groups)."""
    rng = random.Random(top)
    hist = [rng.choice([0, 3, 62, 63, 64, 129, 700]) for _ in range(11)]
    new = [rng.randint(0, top) for _ in hist]
    new[3] = top
    x = Batch(heads, kv, dim, 16 if top == 4 else 64, hist, new, seed=top, pad_rows=1)
    out, b = run_attention(x)
    b.check()
    check_rows(x, out)


@pytest.mark.parametrize("heads,kv,dim", HEADS)
@pytest.mark.parametrize("page", [16, 64, 128])
def test_many_new_tokens(heads, kv, dim, page):
    """Prompts and chunks of odd lengths next to single tokens and an idle sequence."""
    hist = [0, 0, 130, 1000, 513, 77, 0]
    new = [1, 300, 257, 1, 128, 0, 43]
    x = Batch(heads, kv, dim, page, hist, new, seed=page, pad_rows=2, packed=page == 16)
    out, b = run_attention(x)
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
    out, b = run_attention(x, window)
    b.check()
    x.table = keep
    check_rows(x, out, window)


def prefix_launches(b, run):
    """How many prefix launches a call of run() makes."""
    before = b.timing_table().get("attn_paged_prefix", (0, 0))[1]
    b.timing(True)
    out = run()
    b.timing_collect()
    b.timing(False)
    return out, b.timing_table().get("attn_paged_prefix", (0, 0))[1] - before


def shared_prefix(heads, kv, dim, prefix, page, top, seqs, own_launch):
    """seqs sequences behind one prefix, some of which hold nothing else; table entries for
    the prefix are junk.  The prefix gets a launch of its own where that pays."""
    rng = random.Random(prefix + top)
    hist = [prefix + (0, 1, 17, 64, 100, 300, 0)[i % 7] for i in range(seqs)]
    new = [rng.randint(1, top) for _ in hist]
    new[4] = 0
    x = Batch(heads, kv, dim, page, hist, new, seed=top, prefix=prefix, pad_rows=2)
    keep = x.table.clone()
    x.table[:, :prefix // page] = -3
    b = block(heads, kv, dim)
    (out, _), n = prefix_launches(b, lambda: run_attention(x, max_new=top))
    b.check()
    assert n == own_launch
    x.table = keep
    check_rows(x, out)


@pytest.mark.parametrize("heads,kv,dim", HEADS)
@pytest.mark.parametrize("prefix,page", [(16, 16), (128, 64), (1040, 16)])
@pytest.mark.parametrize("top", [1, 3, 150])
def test_short_shared_prefix(heads, kv, dim, prefix, page, top):
    shared_prefix(heads, kv, dim, prefix, page, top, 7, 0)


@pytest.mark.parametrize("heads,kv,dim,prefix,page,top,seqs", [
    (12, 2, 128, 1040, 16, 1, 130), (12, 2, 128, 4096, 64, 4, 40), (12, 2, 128, 7056, 16, 30, 70),
    (32, 2, 128, 2064, 16, 1, 70), (32, 2, 128, 9600, 128, 2, 30), (4, 2, 64, 2048, 32, 1, 100),
    (16, 16, 64, 2064, 16, 1, 16), (16, 16, 64, 2048, 128, 9, 16), (16, 16, 64, 3088, 16, 40, 20),
    (8, 4, 128, 2080, 32, 1, 60), (32, 8, 64, 2064, 16, 5, 30), (16, 2, 64, 4128, 32, 1, 40)])
def test_long_shared_prefix(heads, kv, dim, prefix, page, top, seqs):
    shared_prefix(heads, kv, dim, prefix, page, top, seqs, 1)


def test_shared_prefix_equals_the_same_batch_without_it():
    x = Batch(12, 2, 128, 64, [2048 + h for h in (0, 5, 70, 300)] * 20, [1, 2, 1, 3] * 20, seed=4,
              prefix=2048)
    b = block(12, 2, 128)
    (a, _), n = prefix_launches(b, lambda: run_attention(x))
    (c, _), m = prefix_launches(b, lambda: run_attention(x, prefix_pages=None))
    b.check()
    assert (n, m) == (1, 0)
    check_rows(x, a)
    check_rows(x, c)


@pytest.mark.parametrize("hist,new", [([20000], [1]), ([9000, 3], [1, 4]), ([5000], [700])])
def test_one_long_sequence_is_cut_over_the_gpu(hist, new):
    x = Batch(12, 2, 128, 64, hist, new, seed=1)
    out, b = run_attention(x)
    b.check()
    check_rows(x, out)


def test_many_short_sequences():
    """More sequences than CTAs; units wholly inside one CTA."""
    rng = random.Random(5)
    hist = [rng.randint(0, 70) for _ in range(1500)]
    x = Batch(4, 2, 64, 16, hist, [1] * 1500, seed=5)
    out, b = run_attention(x)
    b.check()
    check_rows(x, out)


@pytest.mark.parametrize("heads,kv,dim,top", [(16, 1, 64, 2), (12, 2, 128, 2), (8, 4, 128, 1)])
def test_short_pieces_one_after_another_give_the_same_bits(heads, kv, dim, top):
    """Every tile ends a piece: a warp is in the next piece's maxima while another still
    finishes the one before."""
    rng = random.Random(21)
    hist = [rng.randint(0, 62) for _ in range(2000)]
    x = Batch(heads, kv, dim, 32, hist, [rng.randint(1, top) for _ in hist], seed=21)
    first, b = run_attention(x)
    b.check()
    check_rows(x, first)
    for _ in range(20):
        out, _ = run_attention(x)
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("top", [1, 5, 60])
def test_a_workspace_keeps_nothing_of_the_call_before(top):
    """The same workspace for batches whose sequences are cut over many CTAs, idle, inside
    one CTA, refused, more, fewer."""
    b = block(12, 2, 128)
    nb = b.attn_paged_workspace_bytes(2000, 400)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    for seed, (hist, new) in enumerate([
            ([6000] * 6, [top] * 6), ([6000] * 6, [0, top, 0, 0, 1, 0]),
            ([3] * 152, [1] * 152), ([700] * 153, [0, 1, 1] * 51), ([9000, 2, 4000], [1, top, 0]),
            ([9000], [top]), ([0] * 6, [0] * 5 + [1]), ([800] * 4, [1, 1, top, 1])]):
        x = Batch(12, 2, 128, 64, hist, new, seed=30 + seed, pad_rows=1)
        bad = [1] if len(hist) == 4 else []
        d = x.descriptor(b, max_new=max(new + [1]))
        if bad:
            x.lens[1] = -1
        out = torch.full((x.rows, 12, 128), MARK, dtype=torch.float16, device="cuda")
        b.attn_paged(d, x.q, x.k_pages, x.v_pages, out, ws)
        if bad:
            with pytest.raises(blk.BlkError):
                b.check()
        else:
            b.check()
        check_rows(x, out, skip=bad)


@pytest.mark.parametrize("top", [1, 4, 40])
@pytest.mark.parametrize("prefix", [0, 8192])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_row_of_nan_stays_nan_and_alone(top, prefix, value):
    """A query that is not finite, in a sequence inside one CTA and in one cut over many
    (an infinite score's weight is 2^(inf - inf))."""
    hist = [prefix + h for h in (3, 9000, 500)] * (1 if prefix == 0 else 30)
    x = Batch(12, 2, 128, 64, hist, [top, 1, top] * (len(hist) // 3), seed=22, prefix=prefix)
    want, bound = x.reference()
    x.q[0, 3] = value
    x.q[top, 7] = value
    x.q[2 * top, 11] = value
    out, b = run_attention(x)
    b.check()
    off, bad = (out.double() - want).abs() <= bound, torch.zeros(x.rows, 12, dtype=torch.bool)
    bad[0, 3] = bad[top, 7] = bad[2 * top, 11] = True
    assert out[bad].isnan().all() and off[~bad].all()


@pytest.mark.parametrize("top", [1, 100])
def test_scores_of_any_size(top):
    """Rows whose scores reach +-1000: the running maximum keeps every weight in range."""
    x = Batch(12, 2, 128, 64, [700, 64], [top, 1], seed=6)
    x.q[0] *= 40.0
    x.q[-1] *= 0.0
    out, b = run_attention(x)
    b.check()
    want, _ = x.reference()
    got = out.double()
    assert torch.isfinite(got).all()
    # scores of 40 times the size have 40 times the absolute error (2^-13 * 40 of A);
    # an all-zero q is the mean of V
    v_max = 6.0
    assert ((got[0] - want[0]).abs() <= (2.0 ** -10 + 40 * 2.0 ** -13) * v_max).all()
    assert ((got[-1] - want[-1]).abs() <= 2.0 ** -10 * v_max).all()


def test_offsets_past_32_bits():
    """A pool of 2^32 elements and more: pages at its end."""
    n_pages = (1 << 32) // (2 * 128 * 128) + 5
    x = Batch(12, 2, 128, 128, [300, 4000], [1, 1], seed=7, n_pages=n_pages, junk=0.0)
    x.table[0, 0] = n_pages - 2
    for pool in (x.k_pages, x.v_pages):
        pool[n_pages - 2] = pool[int(x.table[0, 1])]
    out, b = run_attention(x)
    b.check()
    check_rows(x, out)
    # and the append there
    slots = torch.tensor([(n_pages - 1) * 128 + 127, (n_pages - 3) * 128], device="cuda")
    k = torch.randn((2, 2, 128), device="cuda").half()
    b.page_append(k, -k, slots, x.k_pages, x.v_pages)
    b.check()
    assert torch.equal(x.k_pages[n_pages - 1, :, 127], k[0])
    assert torch.equal(x.v_pages[n_pages - 3, :, 0], -k[1])


@pytest.mark.parametrize("top", [1, 90])
def test_refused_sequences_leave_their_rows_and_the_others_are_served(top):
    """On the device: a length past max_len, a row range that does not fit, fewer slots
    than the prefix; each is reported and its rows stay as they were."""
    new = [1, top, 1, 2]
    x = Batch(12, 2, 128, 16, [30, 40, 500, 60], new, seed=8)
    out, b = run_attention(x, max_len=40 + top)
    with pytest.raises(blk.BlkError) as e:
        b.check()
    assert e.value.status == blk.BLK_ERR_PAGE
    check_rows(x, out, skip=[i for i, h in enumerate(x.hist) if h + new[i] > 40 + top])
    b.check()                                    # reported once
    x.lens[2] = -4
    out, b = run_attention(x)
    with pytest.raises(blk.BlkError):
        b.check()
    check_rows(x, out, skip=[2])
    for prefix, seqs in ((64, 3), (4096, 60)):
        x = Batch(12, 2, 128, 64, [prefix, prefix + 1, prefix] * (seqs // 3),
                  [1, top if seqs < 9 else 3, 1] * (seqs // 3), seed=9, prefix=prefix)
        short = [i for i in (0, 7, 8, 9, 31, 59) if i < seqs]
        for i in short:
            x.lens[i] = prefix - 1
        out, b = run_attention(x)
        with pytest.raises(blk.BlkError):
            b.check()
        check_rows(x, out, skip=short)


@pytest.mark.parametrize("top", [1, 60])
@pytest.mark.parametrize("bad", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
def test_a_bad_page_reads_as_zeros_and_is_reported(top, bad):
    x = Batch(12, 2, 128, 16, [100, 40], [top, 1], seed=10)
    pg = int(x.table[0, 2])
    x.table[0, 2] = bad
    out, b = run_attention(x)
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
    """Lengths, row ranges and tables are the device's: a graph captured at one step
    replays the next, on its own stream, with the same bits as the call itself."""
    x = Batch(12, 2, 128, 64, [prefix + h for h in (100, 7, 300)], [top, 1, 2], seed=11,
              prefix=prefix)
    y = Batch(12, 2, 128, 64, [prefix + h for h in (220, 64, 1)], [1, 2, top], seed=12,
              prefix=prefix)
    b = block(12, 2, 128)
    n_pages = max(x.k_pages.shape[0], y.k_pages.shape[0])
    rows, blocks = max(x.rows, y.rows), max(x.max_blocks, y.max_blocks)
    pools = [torch.zeros((n_pages, 2, 64, 128), dtype=torch.float16, device="cuda") for _ in range(2)]
    q = torch.zeros((rows, 12, 128), dtype=torch.float16, device="cuda")
    table = torch.full((3, blocks), -1, dtype=torch.int32, device="cuda")
    lens, start = torch.zeros_like(x.lens), torch.zeros_like(x.row_start)
    pre = torch.zeros(prefix // 64, dtype=torch.int32, device="cuda") if prefix else None
    out = torch.full((rows, 12, 128), MARK, dtype=torch.float16, device="cuda")
    ws = torch.empty(b.attn_paged_workspace_bytes(rows, 3), dtype=torch.uint8, device="cuda")
    d = b.paged_batch(start, lens, table, rows, 64, n_pages, max(2, top), blocks * 64,
                      prefix_pages=pre)

    def load(z):
        for to, src in zip(pools, (z.k_pages, z.v_pages)):
            to[:src.shape[0]] = src
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
            b.attn_paged(d, q, *pools, out, ws, stream=s)
    for z in (x, y, x):
        load(z)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        b.check()
        check_rows(z, out)
        again = torch.full_like(out, MARK)
        b.attn_paged(d, q, *pools, again, ws)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def test_two_streams_with_their_own_workspaces():
    xs = [Batch(12, 2, 128, 64, [2000 + 31 * i, 5, 700], [1, 1 + i % 3, 60 * (i % 2)], seed=20 + i)
          for i in range(4)]
    outs, streams = [], [torch.cuda.Stream() for _ in xs]
    b = block(12, 2, 128)
    args = []
    for x in xs:
        out = torch.full((x.rows, 12, 128), MARK, dtype=torch.float16, device="cuda")
        ws = torch.empty(b.attn_paged_workspace_bytes(x.rows, 3), dtype=torch.uint8, device="cuda")
        args.append((x.descriptor(b), out, ws))
    torch.cuda.synchronize()
    for _ in range(5):
        for x, (d, out, ws), s in zip(xs, args, streams):
            b.attn_paged(d, x.q, x.k_pages, x.v_pages, out, ws, stream=s)
    torch.cuda.synchronize()
    b.check()
    for x, (_, out, _) in zip(xs, args):
        check_rows(x, out)


@pytest.mark.parametrize("top", [2, 90])
@pytest.mark.parametrize("first,width", [(32, 64), (8, 24), (0, 8)])
def test_strided_output_and_the_gaps_between_rows(top, first, width):
    """Rows at 16-byte boundaries only, too."""
    x = Batch(12, 2, 128, 64, [70, 200], [2, top], seed=13)
    wide = torch.full((x.rows, 12 * 128 + width), MARK, dtype=torch.float16, device="cuda")
    out, b = run_attention(x, out=wide[:, first:first + 12 * 128].unflatten(1, (12, 128)))
    b.check()
    check_rows(x, out)
    assert (wide[:, :first] == MARK).all() and (wide[:, first + 12 * 128:] == MARK).all()


@pytest.mark.parametrize("new,prefix", [([1, 3, 1], 0), ([60, 3, 90], 0), ([1, 3, 1] * 40, 4096)])
def test_a_workspace_at_a_16_byte_boundary(new, prefix):
    x = Batch(12, 2, 128, 64, [prefix + h for h in (900, 4000, 0)] * (len(new) // 3), new, seed=15,
              prefix=prefix)
    out, b = run_attention(x, shift=16)
    b.check()
    check_rows(x, out)


@pytest.mark.parametrize("top", [1, 5, 70])
def test_rows_before_the_first_sequence_and_idle_batches(top):
    """Row ranges that begin behind the batch's first rows; no sequence with rows at all."""
    x = Batch(12, 2, 128, 64, [100, 7], [1, top], seed=16, pad_rows=4)
    x.row_start += 3
    x.q[3:3 + x.n] = x.q[:x.n].clone()
    out, b = run_attention(x)
    b.check()
    assert (out[:3] == MARK).all()
    x.q = x.q[3:]
    x.rows -= 3
    check_rows(x, out[3:])
    for prefix in (0, 8192):
        x = Batch(12, 2, 128, 64, [prefix + 5] * 80, [0] * 80, seed=17, prefix=prefix, pad_rows=top)
        out, b = run_attention(x, max_new=top)
        b.check()
        assert (out == MARK).all()


@pytest.mark.parametrize("top", [2, 50])
def test_more_new_tokens_than_announced_are_refused(top):
    x = Batch(12, 2, 128, 64, [100, 7, 30], [1, top, 1], seed=18)
    out, b = run_attention(x, max_new=top - 1)
    with pytest.raises(blk.BlkError) as e:
        b.check()
    assert e.value.status == blk.BLK_ERR_PAGE
    check_rows(x, out, skip=[1])
    # row ranges that run backwards or past the batch
    x.row_start[1] = x.rows + 5
    out, b = run_attention(x)
    with pytest.raises(blk.BlkError):
        b.check()
    assert (out[:1 + top] == MARK).all()


def test_argument_errors():
    x = Batch(12, 2, 128, 64, [70, 200], [1, 2], seed=14, prefix=64)
    b = block(12, 2, 128)
    nb = b.attn_paged_workspace_bytes(x.rows, 2)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    out = torch.full((x.rows, 12, 128), MARK, dtype=torch.float16, device="cuda")
    st = torch.cuda.current_stream().cuda_stream

    def call(expect, handle=b.handle, q=x.q.data_ptr(), q_stride=1536, o_stride=1536,
             ws_bytes=nb, kp=x.k_pages.data_ptr(), **kw):
        d = x.descriptor(b)
        for name, val in kw.items():
            setattr(d, name, val)
        rc = blk.blk_attn_paged(handle, d, q, q_stride, kp, x.v_pages.data_ptr(), out.data_ptr(),
                                o_stride, ws.data_ptr(), ws_bytes, st)
        assert rc == expect, (rc, kw)

    S, A, N = blk.BLK_ERR_SHAPE, blk.BLK_ERR_ALIGN, blk.BLK_ERR_NULL
    call(N, handle=None)
    call(N, q=None)
    call(N, kp=None)
    call(N, row_start=None)
    call(N, cache_lens=None)
    call(N, block_table=None)
    call(N, prefix_pages=None)
    call(A, q=x.q.data_ptr() + 2)
    call(A, q_stride=1540)
    call(A, o_stride=1537)
    call(S, q_stride=1528)
    call(S, o_stride=0)
    call(A, block_table=x.table.data_ptr() + 2)
    call(A, row_start=x.row_start.data_ptr() + 4)
    call(S, page_size=48)
    call(S, page_size=8)
    call(S, n_pages=0)
    call(S, n_pages=1 << 31)
    call(S, n_seqs=0)
    call(S, n_seqs=4097)
    call(S, n_rows=0)
    call(S, n_rows=(1 << 20) + 1)
    call(S, max_new=0)
    call(S, max_new=x.rows + 1)
    call(S, max_len=0)
    call(S, prefix_len=65)
    call(S, prefix_len=-64)
    call(S, prefix_len=4096)
    call(blk.BLK_ERR_CACHE_OVERFLOW, max_len=x.max_blocks * 64 + 1)
    call(blk.BLK_ERR_WORKSPACE, ws_bytes=nb - 1)
    call(S, handle=block(12, 2, 128, 50).handle)        # a prefix and a window
    torch.cuda.synchronize()
    assert (out == MARK).all()
    for rows, seqs in ((0, 1), (1, 0), (1, 4097), ((1 << 20) + 1, 1)):
        assert b.attn_paged_workspace_bytes(rows, seqs) == 0
        assert b.step_paged_workspace_bytes(rows, seqs) == 0
    d = x.descriptor(b)
    for bad in (dict(q=x.q[:1]), dict(q=x.q.float()), dict(out=out.cpu()),
                dict(k=x.k_pages[:-1]), dict(k=x.k_pages.transpose(1, 2))):
        with pytest.raises(blk.BlkError) as e:
            b.attn_paged(d, bad.get("q", x.q), bad.get("k", x.k_pages), x.v_pages,
                         bad.get("out", out), ws)
        assert e.value.status == S
    for bad in (ws.cpu(), torch.empty((nb, 2), dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(blk.BlkError) as e:
            b.attn_paged(d, x.q, x.k_pages, x.v_pages, out, bad)
        assert e.value.status == blk.BLK_ERR_WORKSPACE
    args = b._args                             # tensors of another GPU than the block's
    b._args = (args[0], args[1] + 1, *args[2:])
    try:
        with pytest.raises(blk.BlkError) as e:
            b.attn_paged(d, x.q, x.k_pages, x.v_pages, out, ws)
        assert e.value.status == S
    finally:
        b._args = args
