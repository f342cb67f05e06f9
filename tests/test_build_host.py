"""The build script: the library needs nvcc alone, and the host path of the Python serving calls is
rebuilt when what it was made against changes."""
import builtins
import os
import sys

import pytest
import torch

from test_abi import _build_module


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build module writing into a folder of its own, with g++ and nvcc replaced by a recorder."""
    b = _build_module()
    for name in ("BUILD", "LIBDIR"):
        monkeypatch.setattr(b, name, str(tmp_path / name))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "LIBDIR" / "lib.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "LIBDIR" / "binding.so"))
    b.ran = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        b.ran.append(cmd[0])
        done = Done()
        if cmd[0] == "g++":
            done.returncode = int(getattr(b, "broken", False))
        if not done.returncode:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return done

    monkeypatch.setattr(b.subprocess, "run", run)
    return b


@pytest.fixture
def no_torch(monkeypatch):
    plain = builtins.__import__

    def without(name, *a, **kw):
        if name == "torch" or name.startswith("torch."):
            raise ModuleNotFoundError("No module named 'torch'", name="torch")
        return plain(name, *a, **kw)

    monkeypatch.delitem(sys.modules, "torch")
    monkeypatch.setattr(builtins, "__import__", without)


def test_library_is_built_without_torch(build, no_torch):
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.BINDING) and "g++" not in build.ran


def test_library_is_linked_when_the_binding_fails(build):
    build.broken = True
    with pytest.raises(RuntimeError, match="binding"):
        build.build()
    assert os.path.exists(build.LIB)


def test_binding_is_rebuilt_for_another_torch(build, monkeypatch):
    assert build.build_binding() == build.BINDING and build.ran == ["g++"]
    build.build_binding()
    assert build.ran == ["g++"]                          # current
    monkeypatch.setattr(torch, "__version__", "99.0")
    build.build_binding()
    assert build.ran == ["g++"] * 2
    build.build_binding()
    assert build.ran == ["g++"] * 2
    os.utime(build.BINDING, (0, 0))                      # older than its sources
    build.build_binding()
    assert build.ran == ["g++"] * 3
