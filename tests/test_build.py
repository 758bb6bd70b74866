"""What the in-tree build needs: the C library the CUDA toolkit alone, what is
current nothing at all.  Compilers are stood in for by a function that notes the
commands and makes the file behind -o."""
import sys
import types

import pytest

from video_dit_dense_gb300 import _build


@pytest.fixture
def sandbox(monkeypatch, tmp_path):
    """Build outputs in a folder of their own; the commands that were run."""
    ran = []

    def run(cmd, **_):
        ran.append(cmd)
        failed = cmd[0] == "g++" and getattr(run, "no_headers", False)
        if not failed:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("built")
        return types.SimpleNamespace(returncode=int(failed), stdout="", stderr="no such header" if failed else "")
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libh3attn.so"))
    monkeypatch.setattr(_build, "STEP_LIB", str(tmp_path / "_step.so"))
    monkeypatch.setattr(_build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(_build.subprocess, "run", run)
    return types.SimpleNamespace(ran=ran, run=run, path=tmp_path)


def no_nvcc():
    raise RuntimeError("nvcc not found")


def test_the_c_library_needs_no_torch(sandbox, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch fails
    assert _build.build() == _build.LIB
    assert (sandbox.path / "libh3attn.so").exists() and not (sandbox.path / "_step.so").exists()
    assert len(sandbox.ran) == len(_build.SOURCES) + 1 and all("nvcc" in c[0] for c in sandbox.ran)
    before = len(sandbox.ran)
    assert _build.build() == _build.LIB and len(sandbox.ran) == before  # current


def test_a_torch_without_cuda_is_none(sandbox, monkeypatch):
    import torch
    monkeypatch.setattr(torch.version, "cuda", None)
    _build.build()
    assert all("nvcc" in c[0] for c in sandbox.ran)


def test_what_is_current_needs_no_toolkit(sandbox, monkeypatch):
    _build.build()
    assert {c[0] for c in sandbox.ran} >= {"g++"} and (sandbox.path / "_step.so").exists()
    before = len(sandbox.ran)
    monkeypatch.setattr(_build, "_nvcc", no_nvcc)
    assert _build.build() == _build.LIB and len(sandbox.ran) == before


def test_a_host_path_that_does_not_compile_leaves_the_c_library(sandbox):
    sandbox.run.no_headers = True
    with pytest.raises(RuntimeError, match="step.cpp"):
        _build.build()
    assert (sandbox.path / "libh3attn.so").exists()


def test_each_part_is_rebuilt_by_itself(sandbox):
    _build.build()
    (sandbox.path / "_step.so").unlink()
    del sandbox.ran[:]
    _build.build()
    assert [c[0] for c in sandbox.ran] == ["g++"]
    (sandbox.path / "libh3attn.so.stamp").write_text("another")
    del sandbox.ran[:]
    _build.build()
    assert sandbox.ran and all("nvcc" in c[0] for c in sandbox.ran)


def test_the_host_path_is_loaded_with_the_versions_it_was_built_for(sandbox, monkeypatch):
    """Checked before the file is opened: it would read another torch's objects by this one's layouts."""
    import torch
    import video_dit_dense_gb300 as h3
    _build.build()
    monkeypatch.setattr(h3, "_bound", None)
    monkeypatch.setattr(h3, "load", lambda: None)
    opened = []

    def open_module(*_):
        opened.append(1)
        raise ImportError("opened")
    monkeypatch.setattr(h3.importlib, "import_module", open_module)
    with pytest.raises(ImportError, match="opened"):
        h3._get_step()
    for change in (lambda: monkeypatch.setattr(torch, "__version__", "2.0.0"),
                   lambda: (sandbox.path / "_step.so.stamp").write_text("0123456789abcdef0123")):
        change()
        with pytest.raises(RuntimeError, match="was built for"):
            h3._get_step()
    assert len(opened) == 1
    (sandbox.path / "_step.so").unlink()
    with pytest.raises(RuntimeError, match="missing"):
        h3._get_step()


def test_a_torch_that_does_not_load_is_none(sandbox, monkeypatch):
    class Broken:
        @staticmethod
        def find_spec(name, *_):
            if name == "torch":
                raise OSError("libcudart.so: cannot open shared object file")
    monkeypatch.delitem(sys.modules, "torch", raising=False)
    monkeypatch.setattr(sys, "meta_path", [Broken] + sys.meta_path)
    assert _build.build() == _build.LIB
    assert all("nvcc" in c[0] for c in sandbox.ran)
