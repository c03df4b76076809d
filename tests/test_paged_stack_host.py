"""PagedStack's order on streams, on the host: a stand-in for the streams records on which
one each of the runner's own tensors is made, and in which order streams wait."""
from contextlib import contextmanager
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")
import decode_qwen2_block_gb300 as blk  # noqa: E402
from decode_qwen2_block_gb300 import stack as stack_mod  # noqa: E402


class Stream:
    def __init__(self, name, log):
        self.name, self.log, self.cuda_stream = name, log, 0

    def wait_stream(self, other):
        self.log.append(("wait", self.name, other.name))


class Torch:
    """torch, with streams of the test's own and every tensor made on the CPU."""

    def __init__(self, log):
        self.log = log
        self.now = [Stream("current", log)]
        self.cuda = SimpleNamespace(current_stream=lambda: self.now[-1], stream=self._stream)

    @contextmanager
    def _stream(self, s):
        self.now.append(s)
        yield
        self.now.pop()

    def __getattr__(self, name):
        real = getattr(torch, name)
        if name not in ("full", "empty", "zeros", "tensor"):
            return real

        def make(*a, **kw):
            self.log.append((name, self.now[-1].name))
            return real(*a, **kw)
        return make


@pytest.fixture
def runner(monkeypatch):
    log = []
    fake = Torch(log)
    monkeypatch.setattr(stack_mod, "torch", fake)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)   # (CUDA tensors' own)
    monkeypatch.setattr(stack_mod, "blk_step_paged_stack",
                        lambda *a: log.append(("layers", fake.now[-1].name)) or blk.BLK_OK)

    class Block:
        handle = None

        def __init__(self, shape, max_ctx, chain=False):
            pass

        weights = staticmethod(lambda w: blk.BlkWeights())

        def step_paged_workspace_bytes(self, rows, seqs):
            return 64

        def page_plan(self, page, lens, news, free, table, start, slots, pos, used, stream=None):
            log.append(("plan", fake.now[-1].name))
            for b in range(len(lens)):                      # (one sequence of whole pages)
                table[b, :free.numel()] = free

        def paged_batch(self, *a, **kw):
            return None

        def _paged_rows(self, *a):
            pass

    monkeypatch.setattr(stack_mod, "Block", Block)
    shape = SimpleNamespace(n_kv_heads=2, head_dim=64, hidden=8)
    pg = stack_mod.PagedStack(shape, [{}], 64, 12, 16, 3, 64, device="cpu")
    del log[:]
    return pg, fake, log


def test_a_prefix_is_computed_wholly_on_its_stream(runner):
    """The last step's stream is given again while another one is current: nothing waits
    between those two, so no tensor of the step may be made on the current one."""
    pg, fake, log = runner
    pg._last = other = Stream("other", log)
    pg.prefill_prefix(torch.zeros(32, 8), stream=other)
    assert log and {e[1] for e in log if e[0] != "wait"} == {"other"}
    assert pg.prefix.tolist() == [0, 1] and pg.table[:, :2].tolist() == [[0, 1]] * 3


def test_a_prefix_on_a_new_stream_follows_the_last_one_from_its_first_tensor_on(runner):
    pg, fake, log = runner
    pg.prefill_prefix(torch.zeros(32, 8), stream=Stream("new", log))
    assert log[0] == ("wait", "new", "current")
    assert {e[1] for e in log if e[0] != "wait"} == {"new"}


def test_the_prefix_holds_no_other_memory(runner):
    """The pages alone are kept, not the table that they were planned in."""
    pg, fake, log = runner
    pg.prefill_prefix(torch.zeros(32, 8))
    assert pg.prefix.untyped_storage().nbytes() == 2 * 4


def test_steps_wait_for_the_step_before_on_another_stream(runner):
    pg, fake, log = runner
    a, b = Stream("a", log), Stream("b", log)
    for s in (a, a, b, None):
        pg.step(torch.zeros(2, 8), [2], stream=s)
    assert [e for e in log if e[0] == "wait"] == [("wait", "a", "current"), ("wait", "b", "a"),
                                                 ("wait", "current", "b")]


def test_the_runners_buffers_are_held_for_every_stream_that_steps_use(runner, monkeypatch):
    """A buffer whose memory the allocator gives to another tensor once the runner is gone,
    while a step on a stream not its own still runs, is recorded for that stream; each once."""
    pg, fake, log = runner
    held = []
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: held.append((t.data_ptr(), s.name)))
    own = [t.data_ptr() for pair in pg.pools for t in pair] + [pg.table.data_ptr(), pg.ws.data_ptr()]
    a, b = Stream("a", log), Stream("b", log)
    pg.step(torch.zeros(2, 8), [2])
    assert held == []
    pg.step(torch.zeros(2, 8), [2], stream=a)
    assert sorted(held) == sorted((p, "a") for p in own)
    pg.step(torch.zeros(2, 8), [2], stream=a)
    pg.step(torch.zeros(2, 8), [2])
    assert len(held) == len(own)
    pg.free(0)
    pg.prefill_prefix(torch.zeros(32, 8), stream=b)
    del held[:]
    pg.step(torch.zeros(2, 8), [2], stream=a)     # (the prefix is newer than a's first step)
    pg.step(torch.zeros(2, 8), [2], stream=b)
    assert held == [(pg.prefix.data_ptr(), "a")]
