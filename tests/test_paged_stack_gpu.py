"""GPU tests of PagedStack's runner across streams."""
import pytest
import torch

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
