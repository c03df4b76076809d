"""The build: the library needs nothing of Python's, the module of the paged calls is
built anew for another Python or torch.  On the host, with the compilers stood in for."""
import os

import pytest

from decode_qwen2_block_gb300 import build as gpu_build


@pytest.fixture
def tools(monkeypatch, tmp_path):
    """An empty build folder, and compilers that write their output file alone."""
    calls = []

    def run(cmd, what, verbose=False):
        calls.append(cmd)
        if "binding.cpp" in what and getattr(run, "fail", False):
            raise RuntimeError(what)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("x")

    monkeypatch.setattr(gpu_build, "_run", run)
    monkeypatch.setattr(gpu_build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(gpu_build, "LIB", str(tmp_path / "libblk.so"))
    monkeypatch.setattr(gpu_build, "NATIVE", str(tmp_path / "_native.so"))
    monkeypatch.setattr(gpu_build, "NATIVE_TAG", str(tmp_path / "_build" / "native.tag"),
                        raising=False)
    return run, calls


@pytest.fixture
def no_torch(monkeypatch):
    real = gpu_build.importlib.util.find_spec
    monkeypatch.setattr(gpu_build.importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else real(name, *a))


def test_without_torch_the_library_is_built_alone(tools, no_torch):
    _, calls = tools
    assert gpu_build.build() == gpu_build.LIB
    assert os.path.exists(gpu_build.LIB) and not os.path.exists(gpu_build.NATIVE)
    n = len(calls)
    gpu_build.build()                          # and is up to date without the module
    assert len(calls) == n


def test_a_module_that_cannot_be_built_leaves_the_library(tools):
    run, _ = tools
    run.fail = True
    with pytest.raises(RuntimeError, match="binding"):
        gpu_build.build()
    assert os.path.exists(gpu_build.LIB)


def test_the_module_is_built_anew_for_another_torch(tools, monkeypatch):
    _, calls = tools
    gpu_build.build()
    assert os.path.exists(gpu_build.NATIVE)
    n = len(calls)
    gpu_build.build()
    assert len(calls) == n
    real = gpu_build.importlib.metadata.version
    monkeypatch.setattr(gpu_build.importlib.metadata, "version",
                        lambda name: "0.0.1" if name == "torch" else real(name))
    gpu_build.build()
    new = calls[n:]
    assert len(new) == 2 and all(c[0] == "g++" for c in new)      # the module, not the kernels
    gpu_build.build()
    assert len(calls) == n + 2
