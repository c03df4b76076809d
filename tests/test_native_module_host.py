"""The compiled module of the paged calls: who needs it, and who does not.  On the host."""
import importlib
import sys
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")
import decode_qwen2_block_gb300 as blk  # noqa: E402

MODULE = "decode_qwen2_block_gb300._native"
SHAPE = SimpleNamespace(hidden=128, n_heads=2, n_kv_heads=1, head_dim=64, intermediate=128,
                        has_qkv_bias=False, rms_eps=1e-6, rope_theta=1e4)


@pytest.fixture
def no_gpu(monkeypatch):
    """Null handles, which need no GPU."""
    monkeypatch.setattr(blk, "blk_create", lambda cfg: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


@pytest.fixture
def no_module(monkeypatch):
    monkeypatch.setitem(sys.modules, MODULE, None)      # importing it fails
    monkeypatch.delattr(blk, "_native", raising=False)
    monkeypatch.setattr(blk, "_calls", None, raising=False)


def test_a_block_needs_the_module_for_the_paged_calls_alone(no_gpu, no_module):
    b = blk.Block(SHAPE, 64)
    t = torch.zeros(1, dtype=torch.int64)
    for call in (lambda: b.page_plan(16, t, None, t, t, t, t, t, t),
                 lambda: b.page_append(t, t, t, t, t), lambda: b.attn_paged(t, t, t, t, t, t)):
        with pytest.raises(ImportError):
            call()


def test_the_module_is_loaded_with_the_first_paged_call(no_gpu, monkeypatch):
    monkeypatch.setattr(blk, "_calls", None)
    b = blk.Block(SHAPE, 64)
    t = torch.zeros(1, dtype=torch.int64)
    for _ in range(2):
        with pytest.raises(blk.BlkError) as e:          # (a CPU tensor)
            b.page_plan(16, t, None, t, t, t, t, t, t)
        assert e.value.status == blk.BLK_ERR_SHAPE
    assert blk._calls is importlib.import_module(MODULE)


def test_the_module_calls_the_library_that_is_loaded(tmp_path):
    """With a library of another place loaded, the in-tree one (whose kernels and handles are
    others) does not come in beside it."""
    import os
    import shutil
    import subprocess
    other = str(tmp_path / "libother.so")
    shutil.copy(blk.LIB_PATH, other)
    code = ("import sys, torch, decode_qwen2_block_gb300 as blk; blk.load(sys.argv[1]); blk._paged_calls();"
            "print(open('/proc/self/maps').read())")
    root = os.path.dirname(os.path.dirname(blk.LIB_PATH))
    maps = subprocess.run([sys.executable, "-c", code, other], cwd=root, check=True,
                          capture_output=True, text=True).stdout
    assert other in maps and "_native" in maps and "libblk.so" not in maps


def test_the_module_refuses_calls_before_it_has_a_library():
    """(in a process of its own: the module is bound once)"""
    import os
    import subprocess
    code = ("import torch; from decode_qwen2_block_gb300 import _native\n"
            "try: _native.bind(0, 0, 0)\n"
            "except ValueError: print('refused')")
    root = os.path.dirname(os.path.dirname(blk.LIB_PATH))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr
