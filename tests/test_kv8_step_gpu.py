"""GPU tests of a block step over 8-bit pages: the new slots bit for bit what the append
makes of the fp16 step's K/V, every row against the oracle's forward of that row over the
values that the slots before it stand for, and the runner."""
import numpy as np
import pytest
import torch

import decode_qwen2_block_gb300 as blk
import oracle
import synth
from decode_qwen2_block_gb300.stack import LayerStack, PagedStack
from gpu_harness import assert_close, to_dev
from kv8_reference import BLOCK, quantise, same, values

pytestmark = pytest.mark.gpu
E5 = torch.float8_e5m2


def _i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


def _pools8(n_pages, kv, page, dim, fill=0):
    def make(last):
        return torch.full((n_pages, kv, page, last), fill, dtype=torch.uint8, device="cuda")
    return [make(dim), make(dim), make(dim // BLOCK).view(E5), make(dim // BLOCK).view(E5)]


def _flat(t):
    return t.view(torch.uint8).transpose(1, 2).reshape(-1, t.shape[1], t.shape[3])


def _check_step(s, page, hist, new, seed, window=0, prefix=0, rows_checked=None, pad=2):
    """Histories quantised into pages, one step, and the checks.  The oracle takes one row at a
    time over the values of the slots before it; the row's own slot it holds in fp16."""
    C = max(h + t for h, t in zip(hist, new)) + 1
    B, n, kv, dim = len(hist), sum(new), s.n_kv_heads, s.head_dim
    w = synth.block_weights(s, seed=seed)
    wd = {k: to_dev(v) for k, v in w.items()}
    block = blk.Block(s, C)
    block.set_window(window)
    caches = [synth.kv_history(s, C, h, layer=b, seed=seed) for b, h in enumerate(hist)]
    for k, v in caches[1:]:
        k[:, :prefix], v[:, :prefix] = caches[0][0][:, :prefix], caches[0][1][:, :prefix]
    first = prefix // page
    n_pages = first + sum(-(-(h + t) // page) - first for h, t in zip(hist, new)) + 4
    ids = np.random.default_rng(seed).permutation(n_pages).astype(np.int32)
    table = torch.full((B, -(-C // page) + 1), -1, dtype=torch.int32, device="cuda")
    pools = _pools8(n_pages, kv, page, dim, 0x7f)      # (unwritten blocks are NaN)
    pools16 = [torch.zeros((n_pages, kv, page, dim), dtype=torch.float16, device="cuda")
               for _ in range(2)]
    table[:, :first] = to_dev(ids[:first])
    at = first
    for b, h in enumerate(hist):
        k = -(-h // page) - first
        table[b, first:first + k] = to_dev(ids[at:at + k])
        at += k
        if h:
            slot = torch.arange(h, device="cuda")
            slots = table[b, slot // page].long() * page + slot % page
            kd, vd = (to_dev(c[:, :h]).transpose(0, 1) for c in caches[b])
            block.page_append_kv8(kd, vd, slots, *pools)
            block.page_append(kd, vd, slots, *pools16)
    rows = n + pad
    start, slots, pos, used = (torch.empty(k, dtype=torch.int64, device="cuda")
                               for k in (B + 1, rows, rows, 1))
    block.page_plan(page, _i64(hist), _i64(new), to_dev(ids[at:]), table, start, slots, pos, used)
    before = [_flat(p).clone() for p in pools]
    x = synth.hidden_input(s, rows, seed=seed, stream_offset=3)
    batch = block.paged_batch(start, _i64(hist), table, rows, page, n_pages, max(new), C,
                              prefix_pages=to_dev(ids[:first]) if prefix else None)
    ws = torch.full((block.step_paged_workspace_bytes(rows, B, prefix=prefix > 0),), 255,
                    dtype=torch.uint8, device="cuda")
    out = torch.empty((rows, s.hidden), dtype=torch.float16, device="cuda")
    out16 = torch.empty_like(out)
    wt = blk.Block.weights(wd)
    block.step_paged_kv8(wt, batch, to_dev(x), pos, slots, *pools, out, ws)
    block.step_paged(wt, batch, to_dev(x), pos, slots, *pools16, out16, ws)
    torch.cuda.synchronize()
    block.check()
    sl = slots[:n]
    # new slots: the append of the fp16 step's K/V; all others as they were
    k16, v16 = (p.transpose(1, 2).reshape(-1, kv, dim)[sl] for p in pools16)
    for rows16, codes, scales, b_codes, b_scales in ((k16, pools[0], pools[2], before[0], before[2]),
                                                     (v16, pools[1], pools[3], before[1], before[3])):
        c, sc = quantise(rows16)
        b_codes[sl], b_scales[sl] = c, sc
        assert torch.equal(_flat(codes), b_codes) and torch.equal(_flat(scales), b_scales)
    # rows against the oracle, over what the slots before them stand for
    val_k, val_v = (values(_flat(pools[i]), _flat(pools[i + 2])).half().cpu().numpy() for i in range(2))
    tab, got, r = table.cpu().numpy(), out.cpu().numpy(), 0
    for b, (h, t) in enumerate(zip(hist, new)):
        sl_b = [tab[b, j // page] * page + j % page for j in range(h + t)]
        for j in range(t):
            if rows_checked is None or (b, j) in rows_checked:
                kc, vc = np.zeros((kv, C, dim), np.float16), np.zeros((kv, C, dim), np.float16)
                kc[:, :h + j] = val_k[sl_b[:h + j]].transpose(1, 0, 2)
                vc[:, :h + j] = val_v[sl_b[:h + j]].transpose(1, 0, 2)
                o, _, _ = oracle.block_forward(s, w, x[r + j:r + j + 1], [h + j], h + j, kc, vc, window=window)
                assert_close(got[r + j:r + j + 1], o, f"sequence {b} row {j}")
        r += t


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("new", [[1, 1, 1, 1, 1], [3, 0, 1, 5, 2], [40, 1, 70, 0, 33]])
def test_tiny_step(page, new):
    _check_step(synth.TINY, page, [0, 37, 64, 100, 15], new, seed=21)


def test_tiny_step_of_many_sequences():
    """More than 128 rows: K/V through the projection's epilogue and the append."""
    rng = np.random.default_rng(22)
    hist = [int(v) for v in rng.integers(0, 90, size=150)]
    _check_step(synth.TINY, 32, hist, [1] * 150, seed=22, rows_checked={(b, 0) for b in range(0, 150, 7)})


@pytest.mark.parametrize("new", [[1, 1, 1], [5, 4, 1], [90, 1, 60]])
def test_1p5b_step(new):
    _check_step(synth.QWEN2_1P5B, 64, [1000, 17, 300], new, seed=23,
                rows_checked={(b, j) for b in range(3) for j in (0, new[b] - 1)})


@pytest.mark.parametrize("new", [[1, 2, 1], [50, 1, 3]])
def test_windowed_step(new):
    _check_step(synth.TINY, 16, [200, 31, 5], new, seed=25, window=33)


@pytest.mark.parametrize("new", [[1, 1, 2, 1], [1, 60, 2, 1]])
def test_step_behind_a_shared_prefix(new):
    _check_step(synth.TINY, 32, [96, 100, 160, 97], new, seed=26, prefix=96)


def _layers(s, n, seed):
    return [{k: to_dev(v) for k, v in synth.block_weights(s, layer=l, seed=seed).items()}
            for l in range(n)]


def test_stack_equals_one_call_per_layer():
    s, n, page, new = synth.TINY, 3, 16, [5, 1, 40]
    wd = _layers(s, n, 31)
    x = to_dev(synth.hidden_input(s, sum(new), seed=31))
    st = PagedStack(s, wd, 128, 40, page, 3, 64, kv8=True)
    out = st.step(x, new)
    block = blk.Block(s, 128)
    start, lens = _i64([0, 5, 6, 46]), _i64([0, 0, 0])
    slot = torch.cat([torch.arange(t, device="cuda") for t in new])
    seq = torch.repeat_interleave(torch.arange(3, device="cuda"), _i64(new))
    slots = st.table[seq, slot // page].long() * page + slot % page
    batch = block.paged_batch(start, lens, st.table, sum(new), page, 40, 40, 128)
    ws = torch.empty(block.step_paged_workspace_bytes(64, 3), dtype=torch.uint8, device="cuda")
    cur = x
    for l in range(n):
        pools = _pools8(40, s.n_kv_heads, page, s.head_dim)
        nxt = torch.empty_like(x)
        block.step_paged_kv8(blk.Block.weights(wd[l]), batch, cur, slot, slots, *pools, nxt, ws)
        for a, b in zip(pools, st.pools[l]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        cur = nxt
    torch.cuda.synchronize()
    block.check()
    st.block.check()
    assert torch.equal(cur.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("prefix", [0, 32])
@pytest.mark.parametrize("kv8", [False, True])
def test_read_gives_the_caches_and_a_contiguous_stack_goes_on_from_them(prefix, kv8):
    """Requests through prompts, chunks and tokens; what ``read`` gives is what the slots stand
    for, and a request moved to contiguous caches goes on as it does over pages (its next
    token's own K/V are fp16 there, rounded to 2^-8 of a block's greatest magnitude here)."""
    s, n, C, page = synth.TINY, 2, 256, 16
    wd = _layers(s, n, 33)
    pg = PagedStack(s, wd, C, 30, page, 3, 160, kv8=kv8)
    feed = to_dev(synth.hidden_input(s, 400, seed=33))
    at = 0
    if prefix:
        pg.prefill_prefix(feed[:prefix])
        at = prefix
    for new in ([50, 7, 0], [1, 60, 33], [4, 1, 2]):
        pg.step(feed[at:at + sum(new)], new)
        at += sum(new)
    pg.block.check()
    for b in range(3):
        got = pg.read(b)
        L = pg.lens[b]
        slot = torch.arange(L, device="cuda")
        pages = pg.table[b][slot // page].long()
        for pool, (k, v) in zip(pg.pools, got):
            for i, t in enumerate((k, v)):
                assert t.shape == (s.n_kv_heads, L, s.head_dim)
                if kv8:
                    want = values(_flat(pool[i]), _flat(pool[i + 2]))[pages * page + slot % page]
                else:
                    want = pool[i][pages, :, slot % page]
                assert same(t, want.transpose(0, 1))
    L = pg.lens[1]
    ref = LayerStack(s, wd, C, 16)
    pg.read(1, caches=ref.caches)
    x = feed[at:at + 1]
    want = ref.run("decode", x, _i64([L]), L).clone()
    out = pg.step(torch.cat((x, x, x)), [1, 1, 1])
    assert_close(out[1:2].cpu().numpy(), want.cpu().numpy(), "the next token")
    with pytest.raises(blk.BlkError):
        pg.read(1, caches=ref.caches[:1])
    with pytest.raises(blk.BlkError):
        pg.read(1, caches=[(k[:, :3], v[:, :3]) for k, v in ref.caches])


def test_steps_on_changing_streams():
    s = synth.TINY
    wd = _layers(s, 3, 37)
    x = to_dev(synth.hidden_input(s, 200, seed=37))
    news = [[40, 3], [1, 20], [1, 1], [30, 1], [1, 1]]
    torch.cuda.synchronize()
    results = []
    for many in (False, True):
        streams = [torch.cuda.Stream() for _ in range(3)] if many else [torch.cuda.current_stream()]
        pg = PagedStack(s, wd, 128, 30, 16, 2, 64, kv8=True)
        at, outs = 0, []
        for i, new in enumerate(news):
            outs.append(pg.step(x[at:at + sum(new)], new, stream=streams[i % len(streams)]))
            at += sum(new)
        got = pg.read(0, stream=streams[1 % len(streams)])
        torch.cuda.synchronize()
        pg.block.check()
        results.append(torch.cat([t.flatten() for t in (*outs, *got[2])]))
    assert torch.equal(results[0].view(torch.int16), results[1].view(torch.int16))


def test_steps_whose_kernels_overlap_equal_steps_whose_kernels_do_not():
    """The attention begins under the kernel that writes q and the new slots; with the
    per-kernel timing on no two kernels overlap: the same bits."""
    s, n, B = synth.TINY, 6, 60
    wd = _layers(s, n, 38)
    x = to_dev(synth.hidden_input(s, 1800, seed=38))
    prompts = [(37 * b) % 61 + 1 for b in range(B)]
    results = []
    for timed in (False, True):
        pg = PagedStack(s, wd, 256, 900, 16, B, 1800, kv8=True)
        pg.block.timing(timed)
        pg.step(x[:sum(prompts[:20])], prompts[:20])
        pg.block.timing_collect()
        pg.step(x[:sum(prompts[20:])], [0] * 20 + prompts[20:])
        outs = []
        for step in range(40):
            new = [1 + (b + step) % 4 if step % 5 == 4 else 1 for b in range(B)]
            outs.append(pg.step(x[step:step + sum(new)], new))
            pg.block.timing_collect()
        pg.block.timing(False)
        torch.cuda.synchronize()
        pg.block.check()
        results.append(torch.cat(outs))
    assert torch.equal(results[0].view(torch.int16), results[1].view(torch.int16))


@pytest.mark.parametrize("rows", [4, 150])
def test_step_reports_a_slot_outside_the_pool_and_writes_nothing_there(rows):
    s = synth.TINY
    block = blk.Block(s, 256)
    wt = blk.Block.weights(wd := {k: to_dev(v) for k, v in synth.block_weights(s, seed=4).items()})
    whole = _pools8(13, 2, 16, 64, 77)
    pools = [p[1:12] for p in whole]
    table = torch.arange(11, dtype=torch.int32, device="cuda")[None]
    batch = block.paged_batch(_i64([0, rows]), _i64([0]), table, rows, 16, 11, rows, 176)
    x = to_dev(synth.hidden_input(s, rows, seed=4))
    out = torch.empty_like(x)
    ws = torch.empty(block.step_paged_workspace_bytes(rows, 1), dtype=torch.uint8, device="cuda")
    pos = torch.arange(rows, device="cuda")
    slots = pos.clone()
    slots[1], slots[2], slots[3] = 11 * 16, -16, -1
    block.step_paged_kv8(wt, batch, x, pos, slots, *pools, out, ws)
    torch.cuda.synchronize()
    with pytest.raises(blk.BlkError) as e:
        block.check()
    assert e.value.status == blk.BLK_ERR_PAGE
    for p in whole:
        at = (_flat(p) != 77).any(-1).any(-1).nonzero().flatten().tolist()     # slots written
        assert at == [16] + list(range(16 + 4, 16 + rows))
    assert wd


def test_step_argument_errors_enqueue_nothing():
    s = synth.TINY
    wd = {k: to_dev(v) for k, v in synth.block_weights(s, seed=1).items()}
    block = blk.Block(s, 64)
    pools = _pools8(4, 2, 16, 64, 77)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    batch = block.paged_batch(_i64([0, 2]), _i64([0]), table, 2, 16, 4, 2, 32)
    x = torch.zeros((2, s.hidden), dtype=torch.float16, device="cuda")
    out = torch.empty_like(x)
    pos, slots = _i64([0, 1]), _i64([0, 1])
    ws = torch.empty(block.step_paged_workspace_bytes(2, 1), dtype=torch.uint8, device="cuda")
    wt = blk.Block.weights(wd)
    P = [t.data_ptr() for t in pools]
    A = [t.data_ptr() for t in (x, pos, slots, out, ws)]
    st = torch.cuda.current_stream().cuda_stream

    def call(a=A, p=P, w=wt, nb=ws.numel()):
        return blk.blk_step_paged_kv8(block.handle, w, batch, a[0], a[1], a[2],
                                      blk.BlkKv8Pool(*p) if p else None, a[3], a[4], nb, st)

    for i in range(5):
        assert call([*A[:i], None, *A[i + 1:]]) == blk.BLK_ERR_NULL
        assert call([*A[:i], A[i] + 2, *A[i + 1:]]) == blk.BLK_ERR_ALIGN
    for i in range(4):
        assert call(p=[*P[:i], None, *P[i + 1:]]) == blk.BLK_ERR_NULL
        assert call(p=[*P[:i], P[i] + 8, *P[i + 1:]]) == blk.BLK_ERR_ALIGN
    assert call(p=None) == blk.BLK_ERR_NULL
    assert call(nb=1000) == blk.BLK_ERR_WORKSPACE
    bad = blk.Block.weights(wd)
    bad.w_up = None
    assert call(w=bad) == blk.BLK_ERR_NULL
    for kw in (dict(x=x[:1]), dict(pos=pos.int()), dict(i=0), dict(i=2)):
        q = [t[:-1] if i == kw.get("i") else t for i, t in enumerate(pools)]
        with pytest.raises(blk.BlkError):
            block.step_paged_kv8(wt, batch, kw.get("x", x), kw.get("pos", pos), slots, *q, out, ws)
    torch.cuda.synchronize()
    assert all((p.view(torch.uint8) == 77).all() for p in pools)
