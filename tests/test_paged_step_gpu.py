"""GPU parity of the paged block step: a ragged batch planned on the GPU, its K/V in
pages, every sequence against the oracle's forward of that sequence alone
(relative L2 <= 1e-2, max abs <= 5e-2), its new slots against the oracle's K/V and
every other slot of the pools untouched; and the layer stack's runner over many
steps against the contiguous caches' stack."""
import numpy as np
import pytest
import torch

import decode_qwen2_block_gb300 as blk
import oracle
import synth
from decode_qwen2_block_gb300.stack import LayerStack, PagedStack
from gpu_harness import assert_close, to_dev

pytestmark = pytest.mark.gpu
MARK = -3.5


def _i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


def _check_step(s, page, hist, new, seed, window=0, prefix=0, sample=None, pad=2):
    """Histories moved into pages from contiguous caches, one step, and the checks."""
    C = max(h + t for h, t in zip(hist, new)) + 1
    B, n = len(hist), sum(new)
    w = synth.block_weights(s, seed=seed)
    wd = {k: to_dev(v) for k, v in w.items()}
    block = blk.Block(s, C)
    block.set_window(window)
    caches = [synth.kv_history(s, C, h, layer=b, seed=seed) for b, h in enumerate(hist)]
    for k, v in caches[1:]:                      # the shared prefix's slots are equal
        k[:, :prefix], v[:, :prefix] = caches[0][0][:, :prefix], caches[0][1][:, :prefix]
    first = prefix // page
    n_pages = first + sum(-(-(h + t) // page) - first for h, t in zip(hist, new)) + 4
    ids = np.random.default_rng(seed).permutation(n_pages).astype(np.int32)
    blocks = -(-C // page) + 1
    table = torch.full((B, blocks), -1, dtype=torch.int32, device="cuda")
    pools = [torch.full((n_pages, s.n_kv_heads, page, s.head_dim), MARK, dtype=torch.float16,
                        device="cuda") for _ in range(2)]
    at = first
    table[:, :first] = to_dev(ids[:first])
    for b, h in enumerate(hist):                 # pages of the history, then its slots
        k = -(-h // page) - first
        table[b, first:first + k] = to_dev(ids[at:at + k])
        at += k
        if h:
            slot = torch.arange(h, device="cuda")
            slots = table[b, slot // page].long() * page + slot % page
            kd, vd = (to_dev(c[:, :h]).transpose(0, 1) for c in caches[b])
            block.page_append(kd, vd, slots, *pools)
    free = to_dev(ids[at:])
    rows = n + pad
    start, slots, pos, used = (torch.empty(k, dtype=torch.int64, device="cuda")
                               for k in (B + 1, rows, rows, 1))
    block.page_plan(page, _i64(hist), _i64(new), free, table, start, slots, pos, used)
    before = [p.clone() for p in pools]
    x = synth.hidden_input(s, rows, seed=seed, stream_offset=3)
    batch = block.paged_batch(start, _i64(hist), table, rows, page, n_pages, max(new), C,
                              prefix_pages=to_dev(ids[:first]) if prefix else None)
    ws = torch.full((block.step_paged_workspace_bytes(rows, B, prefix=prefix > 0),), 255,
                    dtype=torch.uint8, device="cuda")
    out = torch.empty((rows, s.hidden), dtype=torch.float16, device="cuda")
    block.step_paged(blk.Block.weights(wd), batch, to_dev(x), pos, slots, *pools, out, ws)
    torch.cuda.synchronize()
    block.check()
    got = out.cpu().numpy()
    sl = slots.cpu().numpy()
    assert (sl[n:] == -1).all()
    r = 0
    new_k, new_v = (p.transpose(1, 2).reshape(-1, s.n_kv_heads, s.head_dim).cpu().numpy()
                    for p in pools)
    for b, (h, t) in enumerate(zip(hist, new)):
        if t and (sample is None or b in sample):
            k, v = caches[b][0].copy(), caches[b][1].copy()
            o, kr, vr = oracle.block_forward(s, w, x[r:r + t], np.arange(h, h + t), h, k, v,
                                             window=window)
            assert_close(got[r:r + t], o, f"sequence {b} out")
            assert_close(new_k[sl[r:r + t]], kr, f"sequence {b} k")
            assert_close(new_v[sl[r:r + t]], vr, f"sequence {b} v")
        r += t
    written = torch.zeros(n_pages * page, dtype=torch.bool, device="cuda")
    written[slots[:n]] = True
    for p, q in zip(pools, before):
        same = (p.view(torch.int16) == q.view(torch.int16)).transpose(1, 2).reshape(
            n_pages * page, -1).all(1)
        assert (same | written).all(), "a slot outside the step's was written"


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("new", [[1, 1, 1, 1, 1], [3, 0, 1, 5, 2], [40, 1, 70, 0, 33]])
def test_tiny_step(page, new):
    _check_step(synth.TINY, page, [0, 37, 64, 100, 15], new, seed=21)


def test_tiny_step_of_many_sequences():
    """More than 128 rows: the projections' 2-SM form, K/V through its epilogue."""
    rng = np.random.default_rng(22)
    hist = [int(v) for v in rng.integers(0, 90, size=150)]
    _check_step(synth.TINY, 32, hist, [1] * 150, seed=22)


@pytest.mark.parametrize("new", [[1, 1, 1], [5, 4, 1], [90, 1, 60]])
def test_1p5b_step(new):
    _check_step(synth.QWEN2_1P5B, 64, [1000, 17, 300], new, seed=23)


def test_gqa4096_step():
    _check_step(synth.GQA_4096, 128, [300, 5], [1, 2], seed=24)


@pytest.mark.parametrize("new", [[1, 2, 1], [50, 1, 3]])
def test_windowed_step(new):
    _check_step(synth.TINY, 16, [200, 31, 5], new, seed=25, window=33)


@pytest.mark.parametrize("new", [[1, 1, 2, 1], [1, 60, 2, 1]])
def test_step_behind_a_shared_prefix(new):
    _check_step(synth.TINY, 32, [96, 100, 160, 97], new, seed=26, prefix=96)


def test_step_argument_errors_enqueue_nothing():
    s = synth.TINY
    w = synth.block_weights(s, seed=1)
    wd = {k: to_dev(v) for k, v in w.items()}
    block = blk.Block(s, 64)
    pools = [torch.full((4, 2, 16, 64), MARK, dtype=torch.float16, device="cuda") for _ in range(2)]
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    batch = block.paged_batch(_i64([0, 2]), _i64([0]), table, 2, 16, 4, 2, 32)
    x = torch.zeros((2, s.hidden), dtype=torch.float16, device="cuda")
    out = torch.empty_like(x)
    pos, slots = _i64([0, 1]), _i64([0, 1])
    ws = torch.empty(block.step_paged_workspace_bytes(2, 1), dtype=torch.uint8, device="cuda")
    wt = blk.Block.weights(wd)
    block.step_paged(wt, batch, x, pos, slots, *pools, out, ws)
    torch.cuda.synchronize()
    for p in pools:
        p.fill_(MARK)
    P = [t.data_ptr() for t in (x, pos, slots, *pools, out, ws)]
    st = torch.cuda.current_stream().cuda_stream
    for i in range(7):
        a = list(P)
        a[i] = None
        assert blk.blk_step_paged(block.handle, wt, batch, *a, ws.numel(), st) == blk.BLK_ERR_NULL
        a[i] = P[i] + 2
        assert blk.blk_step_paged(block.handle, wt, batch, *a, ws.numel(), st) == blk.BLK_ERR_ALIGN
    assert blk.blk_step_paged(block.handle, wt, batch, *P, 1000, st) == blk.BLK_ERR_WORKSPACE
    bad = blk.Block.weights(wd)
    bad.w_up = None
    assert blk.blk_step_paged(block.handle, bad, batch, *P, ws.numel(), st) == blk.BLK_ERR_NULL
    with pytest.raises(blk.BlkError):
        block.step_paged(wt, batch, x[:1], pos, slots, *pools, out, ws)
    with pytest.raises(blk.BlkError):
        block.step_paged(wt, batch, x, pos.int(), slots, *pools, out, ws)
    torch.cuda.synchronize()
    assert all((p == MARK).all() for p in pools)


@pytest.mark.parametrize("rows", [4, 150])
def test_step_reports_a_slot_outside_the_pool_and_writes_nothing_there(rows):
    """Rows whose K/V go to their pages from the projection (few) and by the append."""
    s = synth.TINY
    block = blk.Block(s, 256)
    wt = blk.Block.weights(wd := {k: to_dev(v) for k, v in synth.block_weights(s, seed=4).items()})
    whole = [torch.full((13, 2, 16, 64), MARK, dtype=torch.float16, device="cuda") for _ in range(2)]
    pools = [p[1:12] for p in whole]
    table = torch.arange(11, dtype=torch.int32, device="cuda")[None]
    batch = block.paged_batch(_i64([0, rows]), _i64([0]), table, rows, 16, 11, rows, 176)
    x = to_dev(synth.hidden_input(s, rows, seed=4))
    out = torch.empty_like(x)
    ws = torch.empty(block.step_paged_workspace_bytes(rows, 1), dtype=torch.uint8, device="cuda")
    pos = torch.arange(rows, device="cuda")
    slots = pos.clone()
    slots[1], slots[2], slots[3] = 11 * 16, -16, -1
    block.step_paged(wt, batch, x, pos, slots, *pools, out, ws)
    torch.cuda.synchronize()
    with pytest.raises(blk.BlkError) as e:
        block.check()
    assert e.value.status == blk.BLK_ERR_PAGE
    for p in whole:
        at = (p != MARK).any(-1).any(1).flatten().nonzero().flatten().tolist()     # slots written
        assert at == [16] + list(range(16 + 4, 16 + rows))
    assert wd


def _layers(s, n, seed):
    return [{k: to_dev(v) for k, v in synth.block_weights(s, layer=l, seed=seed).items()}
            for l in range(n)]


def test_stack_equals_one_call_per_layer():
    s, n, page, new = synth.TINY, 3, 16, [5, 1, 40]
    wd = _layers(s, n, 31)
    x = to_dev(synth.hidden_input(s, sum(new), seed=31))
    st = PagedStack(s, wd, 128, 40, page, 3, 64)
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
        pools = [torch.zeros_like(p) for p in st.pools[l]]
        nxt = torch.empty_like(x)
        block.step_paged(blk.Block.weights(wd[l]), batch, cur, slot, slots, *pools, nxt, ws)
        for a, b in zip(pools, st.pools[l]):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        cur = nxt
    torch.cuda.synchronize()
    block.check()
    st.block.check()
    assert torch.equal(cur.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("prefix", [0, 32])
def test_paged_stack_serves_like_contiguous_caches(prefix):
    """Three requests through prompts, chunks, drafts and single tokens, one of them ended
    and replaced: every row as LayerStack computes it on the request's own cache."""
    s, n, C, page = synth.TINY, 2, 256, 16
    wd = _layers(s, n, 33)
    pg = PagedStack(s, wd, C, 30, page, 3, 160)
    refs = [LayerStack(s, wd, C, 128) for _ in range(3)]
    lens = [0, 0, 0]
    feed = synth.hidden_input(s, 2000, seed=33)
    at = 0

    def rows(t):
        nonlocal at
        at += t
        return to_dev(feed[at - t:at])

    def ref(b, x):
        t = x.shape[0]
        o = refs[b].run("prefill" if lens[b] == 0 else "prefill_kv", x,
                        to_dev(synth.positions(lens[b], t)), lens[b]).clone()
        lens[b] += t
        return o

    if prefix:
        x = rows(prefix)
        o = pg.prefill_prefix(x)
        for b in range(3):
            assert_close(o.cpu().numpy(), ref(b, x).cpu().numpy(), "prefix")
    for new in ([50, 7, 0], [1, 60, 33], [1, 1, 1], [4, 1, 2], None, [1, 20, 1], [1, 1, 1]):
        if new is None:                           # request 1 ends, another begins
            held = len(pg.free_ids)
            pg.free(1)
            assert len(pg.free_ids) > held
            lens[1] = 0
            if prefix:
                ref(1, to_dev(feed[:prefix]))
            continue
        x = rows(sum(new))
        out = pg.step(x, new)
        r = 0
        for b, t in enumerate(new):
            if t:
                assert_close(out[r:r + t].cpu().numpy(), ref(b, x[r:r + t]).cpu().numpy(),
                             f"request {b} of {new}")
            r += t
    pg.block.check()
    assert sorted(pg.free_ids + pg.prefix_ids + sum(pg.pages, [])) == list(range(30))


def test_paged_stack_steps_on_changing_streams():
    """Each step on another stream than the last, nothing waiting between them: the bits of
    the same steps on one stream."""
    s = synth.TINY
    wd = _layers(s, 3, 37)
    x = to_dev(synth.hidden_input(s, 200, seed=37))
    news = [[40, 3], [1, 20], [1, 1], [30, 1], [1, 1]]
    torch.cuda.synchronize()
    results = []
    for many in (False, True):
        streams = [torch.cuda.Stream() for _ in range(3)] if many else [torch.cuda.current_stream()]
        pg = PagedStack(s, wd, 128, 30, 16, 2, 64)
        at, outs = 0, []
        for i, new in enumerate(news):
            outs.append(pg.step(x[at:at + sum(new)], new, stream=streams[i % len(streams)]))
            at += sum(new)
        torch.cuda.synchronize()
        pg.block.check()
        results.append(torch.cat(outs))
    assert torch.equal(results[0].view(torch.int16), results[1].view(torch.int16))


def test_steps_whose_kernels_overlap_equal_steps_whose_kernels_do_not():
    """The attention begins under the kernel that writes q and the new slots: the
    projection's finisher, or of more than 128 rows (every fifth step) the append.  With the
    per-kernel timing on no two kernels overlap: the same bits."""
    s, n, B = synth.TINY, 6, 60
    wd = _layers(s, n, 38)
    x = to_dev(synth.hidden_input(s, 1800, seed=38))
    prompts = [(37 * b) % 61 + 1 for b in range(B)]
    results = []
    for timed in (False, True):
        pg = PagedStack(s, wd, 256, 900, 16, B, 1800)
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


def test_paged_stack_refuses_what_does_not_fit():
    s = synth.TINY
    pg = PagedStack(s, _layers(s, 1, 34), 64, 5, 16, 2, 100)
    x = torch.zeros((70, s.hidden), dtype=torch.float16, device="cuda")
    for new, status in (([65], blk.BLK_ERR_CACHE_OVERFLOW), ([50, 20], blk.BLK_ERR_PAGE),
                        ([60, 0, 1], blk.BLK_ERR_SHAPE), ([0, 0], blk.BLK_ERR_SHAPE),
                        ([5, -1], blk.BLK_ERR_SHAPE), ([3], blk.BLK_ERR_SHAPE)):
        m = 70 if new in ([3],) else max(1, sum(t for t in new if t > 0))
        with pytest.raises(blk.BlkError) as e:
            pg.step(x[:m], new)
        assert e.value.status == status, new
    assert pg.lens == [0, 0] and len(pg.free_ids) == 5
    pg.step(x[:64], [64])
    with pytest.raises(blk.BlkError):
        pg.prefill_prefix(x[:16])


def test_generation_over_pages():
    """The serving loop as a whole: embedding, paged stack, LM head, greedy tokens of two
    requests behind one prefix; every step's hidden rows as LayerStack's on the same tokens."""
    s, n, C, vocab = synth.TINY, 2, 128, 300
    wd = _layers(s, n, 35)
    hw = {k: to_dev(v) for k, v in synth.head_weights(vocab, s.hidden, seed=35).items()}
    pg = PagedStack(s, wd, C, 24, 16, 2, 64)
    refs = [LayerStack(s, wd, C, 64) for _ in range(2)]
    b = pg.block
    ws = torch.empty(b.lm_head_workspace_bytes(), dtype=torch.uint8, device="cuda")

    def embed(ids):
        x = torch.empty((len(ids), s.hidden), dtype=torch.float16, device="cuda")
        b.embed(hw["embed"], _i64(ids), x)
        return x

    rng = np.random.default_rng(35)
    prefix = [int(v) for v in rng.integers(0, vocab, 32)]
    prompts = [[int(v) for v in rng.integers(0, vocab, k)] for k in (5, 11)]
    pg.prefill_prefix(embed(prefix))
    fed = [list(prefix) + p for p in prompts]
    out = pg.step(embed(prompts[0] + prompts[1]), [5, 11])
    h = out[[4, 15]].contiguous()
    for step in range(6):
        for i in range(2):
            o = refs[i].run("prefill", embed(fed[i]), _i64(range(len(fed[i]))), 0)
            assert_close(h[i].cpu().numpy(), o[-1].cpu().numpy(), f"request {i} step {step}")
        tok = torch.empty(2, dtype=torch.int64, device="cuda")
        b.lm_head(h, hw["norm_g"], hw["lm_head"], tok, ws)
        nxt = tok.tolist()
        for i in range(2):
            fed[i].append(nxt[i])
        h = pg.step(embed(nxt), [1, 1])
    b.check()
