"""PagedStack over 8-bit pages, on the host: its pools, which call its steps make, and what
``read`` refuses (with stand-ins for the streams and the library's calls)."""
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")
import decode_qwen2_block_gb300 as blk  # noqa: E402
from decode_qwen2_block_gb300 import stack as stack_mod  # noqa: E402
from test_paged_stack_host import Stream, Torch  # noqa: E402


@pytest.fixture
def made(monkeypatch):
    log = []
    fake = Torch(log)
    monkeypatch.setattr(stack_mod, "torch", fake)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)   # (CUDA tensors' own)
    calls = []
    monkeypatch.setattr(stack_mod, "blk_step_paged_stack",
                        lambda *a: calls.append(("fp16", fake.now[-1].name, a)) or blk.BLK_OK)
    monkeypatch.setattr(stack_mod, "blk_step_paged_stack_kv8",
                        lambda *a: calls.append(("kv8", fake.now[-1].name, a)) or blk.BLK_OK)

    class Block:
        handle = None

        def __init__(self, shape, max_ctx, chain=False):
            pass

        weights = staticmethod(lambda w: blk.BlkWeights())

        def step_paged_workspace_bytes(self, rows, seqs):
            return 64

        def page_plan(self, page, lens, news, free, table, start, slots, pos, used, stream=None):
            table[0, :free.numel()] = free

        def paged_batch(self, *a, **kw):
            return None

        def _paged_rows(self, *a):
            pass

        def page_read_kv8(self, slots, kc, vc, ks, vs, k, v, stream=None):
            calls.append(("read", stream.name, (slots.tolist(), k.shape, v.shape)))

    monkeypatch.setattr(stack_mod, "Block", Block)
    shape = SimpleNamespace(n_kv_heads=2, head_dim=64, hidden=8)

    def make(**kw):
        return stack_mod.PagedStack(shape, [{}, {}], 64, 12, 16, 3, 64, device="cpu", **kw)
    return make, calls, log


def test_pools_and_calls(made):
    make, calls, _ = made
    pg = make(kv8=True)
    for p in pg.pools:
        assert [t.dtype for t in p] == [torch.uint8] * 2 + [torch.float8_e5m2] * 2
        assert [t.shape for t in p] == [(12, 2, 16, 64)] * 2 + [(12, 2, 16, 2)] * 2
    pg.step(torch.zeros(3, 8), [3])
    assert [c[0] for c in calls] == ["kv8"]
    arr = calls[0][2][4]
    assert [[getattr(arr[l], f) for f in ("k", "v", "k_scale", "v_scale")] for l in range(2)] == \
        [[t.data_ptr() for t in p] for p in pg.pools]
    make().step(torch.zeros(3, 8), [3])
    assert [c[0] for c in calls] == ["kv8", "fp16"]


def test_read_follows_the_last_step_on_its_own_stream(made):
    make, calls, log = made
    pg = make(kv8=True)
    a = Stream("a", log)
    pg.step(torch.zeros(20, 8), [20], stream=a)
    del calls[:], log[:]
    b = Stream("b", log)
    got = pg.read(0, stream=b)
    assert log[0] == ("wait", "b", "a") and {e[1] for e in log if e[0] != "wait"} == {"b"}
    assert [c[:2] for c in calls] == [("read", "b")] * 2
    assert calls[0][2] == (list(range(20)), (20, 2, 64), (20, 2, 64))
    assert [t.shape for pair in got for t in pair] == [(2, 20, 64)] * 4


def test_read_of_an_empty_sequence_and_refusals(made):
    make, calls, _ = made
    pg = make(kv8=True)
    assert [t.shape for pair in pg.read(1) for t in pair] == [(2, 0, 64)] * 4 and not calls
    pg.step(torch.zeros(5, 8), [5])
    ok = torch.zeros((2, 9, 64), dtype=torch.float16)
    for caches in ([(ok, ok)], [(ok, ok[:, :4])] * 2, [(ok, ok.float())] * 2, [(ok, ok[:1])] * 2,
                   [(ok, ok[..., :32])] * 2):
        with pytest.raises(blk.BlkError) as e:
            pg.read(0, caches=caches)
        assert e.value.status == blk.BLK_ERR_SHAPE
    assert [c[0] for c in calls] == ["kv8"]
    assert pg.read(0, caches=[(ok, ok)] * 2) == [(ok, ok)] * 2
