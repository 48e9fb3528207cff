"""What build() makes, and when: with the compilers replaced by a stand-in that
writes its output file (no GPU, no compilation)."""
import importlib.util
import os
import subprocess
import types

import pytest

from token_verification_gb300 import build


@pytest.fixture
def bench(tmp_path, monkeypatch):
    """build's outputs in a folder of their own, an installed PyTorch of our making, and the
    list of the programs that were run."""
    ran, fail, torch = [], set(), tmp_path / "site" / "torch"
    torch.mkdir(parents=True)
    (torch / "__init__.py").write_text("")
    (torch / "version.py").write_text("1.0")
    for name, at in (("LIB", "libspecverify.so"), ("BINDING", "_binding.so"), ("BUILD", "_build"),
                     ("BUILT_FOR", "_build/binding.txt")):
        monkeypatch.setattr(build, name, str(tmp_path / at))

    def run(cmd, **kw):
        name = os.path.basename(cmd[0])
        ran.append(name)
        if name in fail:
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no " + name)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    have = {"torch": types.SimpleNamespace(origin=str(torch / "__init__.py"))}
    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setattr(build, "nvcc", lambda: "/nowhere/bin/nvcc")
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: have.get(name) if name == "torch" else real(name, *a))
    return types.SimpleNamespace(ran=ran, fail=fail, have=have, torch=torch)


def test_both_once(bench):
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.BINDING)
    assert bench.ran.count("nvcc") == len(build.SOURCES) + 1 and bench.ran.count("g++") == 1
    assert build.up_to_date()
    del bench.ran[:]
    build.build()
    assert bench.ran == []
    build.build(force=True)
    assert bench.ran.count("nvcc") == len(build.SOURCES) + 1 and bench.ran.count("g++") == 1


def test_library_without_pytorch(bench):
    """The C library's users need neither PyTorch nor a binding to it."""
    bench.have.clear()
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert "g++" not in bench.ran and build.up_to_date()


def test_binding_follows_the_installed_pytorch(bench):
    build.build()
    del bench.ran[:]
    (bench.torch / "version.py").write_text("1.1")
    assert not build.up_to_date()
    build.build()
    assert bench.ran == ["g++"] and build.up_to_date()


def test_a_binding_that_fails_leaves_the_library(bench):
    bench.fail.add("g++")
    with pytest.raises(RuntimeError, match="binding"):
        build.build()
    assert os.path.exists(build.LIB) and not build.up_to_date()
    bench.fail.clear()
    del bench.ran[:]
    build.build()
    assert bench.ran == ["g++"]
