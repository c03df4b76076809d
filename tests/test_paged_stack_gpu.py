"""GPU tests of PagedStack's runner across streams, and of steps in a captured graph."""
import ctypes

import pytest
import torch

import decode_qwen2_block_gb300 as blk
import synth
from decode_qwen2_block_gb300.stack import PagedStack
from gpu_harness import to_dev

pytestmark = pytest.mark.gpu


def _layers(s, n, seed):
    return [{k: to_dev(v) for k, v in synth.block_weights(s, layer=l, seed=seed).items()}
            for l in range(n)]


@pytest.mark.parametrize("used_before", [False, True])
def test_a_prefix_on_the_last_stream_while_another_is_current(used_before):
    """The bits of the same calls on one stream, with the current stream busy."""
    s = synth.TINY
    wd = _layers(s, 3, 45)
    x = to_dev(synth.hidden_input(s, 120, seed=45))
    busy = torch.zeros(64 << 20, device="cuda")
    torch.cuda.synchronize()
    results = []
    for apart in (False, True):
        last = torch.cuda.Stream() if apart else torch.cuda.current_stream()
        with torch.cuda.stream(last):
            pg = PagedStack(s, wd, 128, 30, 16, 2, 64)
        if used_before:
            pg.step(x[:20], [20], stream=last)
            pg.free(0)
        if apart:
            for _ in range(20):                  # the current stream is behind by some ms
                busy.add_(1)
        outs = [pg.prefill_prefix(x[20:52], stream=last), pg.step(x[52:60], [3, 5], stream=last),
                pg.step(x[60:62], [1, 1], stream=last)]
        torch.cuda.synchronize()
        pg.block.check()
        assert pg.prefix.tolist() == pg.prefix_ids
        assert pg.table[:, :2].tolist() == [pg.prefix_ids] * 2
        results.append(torch.cat(outs))
    assert torch.equal(results[0].view(torch.int16), results[1].view(torch.int16))


@pytest.mark.parametrize("seqs", [8, 150])
def test_overlapping_kernels_of_the_full_shape(seqs):
    """Steps through blocks of 1536 hidden, whose attention begins under the projection's
    finisher (8 rows) or the append (150): the bits of steps whose kernels do not overlap
    (with the per-kernel timing on)."""
    s = synth.QWEN2_1P5B
    wd = _layers(s, 3, 46)
    x = to_dev(synth.hidden_input(s, 3000, seed=46))
    prompts = [(37 * b) % 15 + 1 for b in range(seqs)]
    prompts[0] = 300
    results = []
    for timed in (False, True):
        pg = PagedStack(s, wd, 512, 700, 16, seqs, 3000)
        pg.block.timing(timed)
        pg.step(x[:sum(prompts)], prompts)
        outs = []
        for step in range(30):
            outs.append(pg.step(x[step:step + seqs], [1] * seqs))
            pg.block.timing_collect()
        pg.block.timing(False)
        torch.cuda.synchronize()
        pg.block.check()
        results.append(torch.cat(outs))
    assert torch.equal(results[0].view(torch.int16), results[1].view(torch.int16))


@pytest.mark.parametrize("rows", [5, 150])
def test_a_captured_step_serves_the_steps_that_follow(rows):
    """Plan and layers captured once, replayed on lengths, tokens and free pages that the
    device holds by then: the bits of the calls themselves, pools included."""
    s, page, n_pages, B, n = synth.TINY, 16, 400, 5, 2
    wd = _layers(s, n, 47)
    block = blk.Block(s, 256)
    w = (blk.BlkWeights * n)(*[blk.Block.weights(d) for d in wd])
    feed = to_dev(synth.hidden_input(s, rows * 12, seed=47)).view(12, rows, -1)
    i64 = dict(dtype=torch.int64, device="cuda")
    results = []
    for captured in (False, True):
        pools = [[torch.zeros((n_pages, s.n_kv_heads, page, s.head_dim), dtype=torch.float16,
                              device="cuda") for _ in range(n)] for _ in range(2)]
        kv = [(ctypes.c_void_p * n)(*[p.data_ptr() for p in side]) for side in pools]
        lens, news = torch.zeros(B, **i64), torch.zeros(B, **i64)
        start, slots, pos, used = (torch.empty(k, **i64) for k in (B + 1, rows, rows, 1))
        table = torch.full((B, 16), -1, dtype=torch.int32, device="cuda")
        free = torch.zeros(60, dtype=torch.int32, device="cuda")
        x = torch.empty_like(feed[0])
        out = torch.empty_like(x)
        ws = torch.empty(block.step_paged_workspace_bytes(rows, B), dtype=torch.uint8, device="cuda")
        batch = block.paged_batch(start, lens, table, rows, page, n_pages, rows, 256)
        stream = torch.cuda.Stream()

        def call():
            block.page_plan(page, lens, news, free, table, start, slots, pos, used, stream=stream)
            rc = blk.blk_step_paged_stack(block.handle, w, n, batch, *kv, x.data_ptr(),
                                          pos.data_ptr(), slots.data_ptr(), out.data_ptr(),
                                          ws.data_ptr(), ws.numel(), stream.cuda_stream)
            assert rc == blk.BLK_OK

        torch.cuda.synchronize()
        if captured:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.stream(stream), torch.cuda.graph(g, stream=stream):
                call()
        taken, outs = 0, []
        for step in range(12):
            new = [(step * 7 + b * 3) % 5 for b in range(B - 1)] + [rows - 30 if step == 0 and rows > 30
                                                                    else 1]
            if sum(new) > rows:
                new = [1] * B
            news.copy_(torch.tensor(new))
            free.copy_(torch.arange(taken, taken + 60) * 37 % n_pages)
            x.copy_(feed[step])
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                g.replay() if captured else call()
            torch.cuda.synchronize()
            block.check()
            taken += int(used)
            lens += news
            outs.append(out[:sum(new)].clone())
        results.append(torch.cat(outs + [p.view(-1, s.hidden) for side in pools for p in side]))
    assert torch.equal(results[0].view(torch.int16), results[1].view(torch.int16))
