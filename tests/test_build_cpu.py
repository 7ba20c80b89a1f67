"""What the build does where torch, or the extension module over its tensors, is missing.

The compilers are stand-ins that write an empty file, or fail.
"""
import importlib.metadata
import os
import types

import pytest

from muon_adamw_hybrid_grad_gb300 import LibraryNotBuilt
from muon_adamw_hybrid_grad_gb300 import build as b


@pytest.fixture
def box(tmp_path, monkeypatch):
    """The build in a folder of its own. box.fail: programs that fail; box.calls: what has been called."""
    box = types.SimpleNamespace(fail=(), calls=[], torch=tmp_path / "torch")
    box.torch.mkdir()
    (box.torch / "__init__.py").write_text("")
    (box.torch / "version.py").write_text("__version__ = '1'")
    monkeypatch.setattr(b, "LIBDIR", str(tmp_path / "lib"))
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(b, "_nvcc", lambda: "/cuda/bin/nvcc")

    def run(cmd, **_):
        name = os.path.basename(cmd[0])
        box.calls.append((name, cmd))
        if name in box.fail:
            return types.SimpleNamespace(returncode=1, stdout="", stderr="Python.h: No such file")
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    def find_spec(name, *_):
        assert name == "torch"
        return types.SimpleNamespace(origin=str(box.torch / "__init__.py")) if box.torch else None

    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b.importlib.util, "find_spec", find_spec)

    def version(name):
        if box.torch is None:
            raise importlib.metadata.PackageNotFoundError(name)
        return "1"

    monkeypatch.setattr(importlib.metadata, "version", version)
    return box


def programs(box):
    names = [name for name, _ in box.calls]
    box.calls.clear()
    return set(names)


def test_library_needs_no_torch(box):
    box.torch = None
    assert os.path.exists(b.build())
    assert programs(box) == {"nvcc"}
    assert not os.path.exists(b.torch_ops_path())
    b.build()
    assert programs(box) == set()


def test_library_needs_no_extension(box):
    """g++ or a header is missing: the library is there all the same, and importing the operators says why they are not."""
    box.fail = ("g++",)
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert os.path.exists(b.build())
    assert not os.path.exists(b.torch_ops_path())
    assert "Python.h" in b.torch_ops_problem()
    box.calls.clear()
    with pytest.warns(RuntimeWarning, match="Python.h"):
        b.build()
    assert programs(box) == {"g++"}  # the library stands, the extension is tried again
    box.fail = ()
    b.build()
    assert programs(box) == {"g++"} and os.path.exists(b.torch_ops_path()) and b.torch_ops_problem() == ""


def test_a_stale_extension_does_not_stay(box):
    b.build()
    assert programs(box) == {"nvcc", "g++"} and os.path.exists(b.torch_ops_path())
    (box.torch / "version.py").write_text("__version__ = '2'")
    box.fail = ("g++",)
    with pytest.warns(RuntimeWarning):
        b.build()
    assert programs(box) == {"g++"} and not os.path.exists(b.torch_ops_path())


def test_another_torch_leaves_the_library(box):
    b.build()
    programs(box)
    b.build()
    assert programs(box) == set()
    (box.torch / "version.py").write_text("__version__ = '2'")
    b.build()
    assert programs(box) == {"g++"}


def test_a_failing_library_still_fails(box):
    box.fail = ("nvcc",)
    with pytest.raises(RuntimeError, match="nvcc failed"):
        b.build()


def test_operators_without_their_extension_say_why(monkeypatch, tmp_path):
    pytest.importorskip("torch")
    b.build()
    from muon_adamw_hybrid_grad_gb300 import ops

    monkeypatch.setattr(b, "torch_ops_path", lambda: str(tmp_path / "_torch_ops.so"))
    monkeypatch.setattr(b, "torch_ops_problem", lambda: "g++ failed: Python.h")
    with pytest.raises(LibraryNotBuilt, match="Python.h"):
        ops._load()
