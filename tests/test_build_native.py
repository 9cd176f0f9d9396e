"""The library and the binding without the native side of the short calls
(_marshal.so): a build in which it fails, one that is stale, and the binding
where it does not load."""

import os
import subprocess
import sys
import types

import pytest
import torch

import gated_deltanet_linear_tree_gb300 as package
from gated_deltanet_linear_tree_gb300 import build, canopy


@pytest.fixture
def empty_tree(tmp_path, monkeypatch):
    """A build folder of its own, with no .cu files; the commands are recorded."""
    for name in ("LIB", "MARSHAL", "MARSHAL_TAG"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "sources", lambda: [])
    done = type("Done", (list,), {"broken": False})()

    def run(cmd, **kw):
        native = "marshal.cpp" in " ".join(cmd)
        done.append("native" if native else "link")
        if native and done.broken:
            return types.SimpleNamespace(returncode=1, stderr="Python.h: No such file or directory")
        with open(cmd[cmd.index("-o") + 1], "w"):
            return types.SimpleNamespace(returncode=0, stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    return done


def test_the_library_is_built_where_the_native_side_is_not(empty_tree):
    empty_tree.broken = True
    with pytest.warns(UserWarning, match="Python.h"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.MARSHAL)
    empty_tree.clear()
    empty_tree.broken = False
    build.build()
    assert empty_tree == ["native"] and os.path.exists(build.MARSHAL)  # and the library is left as it is
    empty_tree.clear()
    build.build()
    assert empty_tree == []


def test_the_native_side_is_built_again_for_another_torch(empty_tree, monkeypatch):
    build.build()
    assert sorted(empty_tree) == ["link", "native"]
    empty_tree.clear()
    monkeypatch.setattr(torch, "__version__", "0.0")
    build.build()
    assert empty_tree == ["native"]


def missing(monkeypatch):
    monkeypatch.setitem(sys.modules, package.__name__ + "._marshal", None)


def other_torch(monkeypatch):
    called = []
    fake = types.SimpleNamespace(built_for="python x, torch 0.0", bind=called.append, step=called.append)
    monkeypatch.setitem(sys.modules, package.__name__ + "._marshal", fake)
    monkeypatch.setattr(package, "_marshal", fake, raising=False)


@pytest.mark.parametrize("case", [missing, other_torch])
def test_the_binding_works_without_the_native_side(monkeypatch, case):
    build.build()
    canopy.load()
    monkeypatch.setattr(canopy, "_lib", None)
    monkeypatch.setattr(canopy, "_marshal", None)
    monkeypatch.delattr(package, "_marshal", raising=False)
    case(monkeypatch)
    with pytest.warns(UserWarning, match="_marshal.so"):
        lib = canopy.load()
    assert lib.canopy_version() == 1 and canopy.prefill_plan(16384, 1, 16, 32, True, 128) == "chunked"
    x = torch.zeros(2, 4, 128)
    with pytest.raises(canopy.CanopyError, match="CUDA"):
        canopy.step(x, x, x, torch.ones(2, 4), torch.ones(2, 4), torch.zeros(2, 4, 128, 128))
