"""fastcall is optional: what keeps it from being built or loaded leaves the library and the calls through ctypes, and a
missing or foreign one is built again although the library is current."""
import os
import subprocess
import sys
import types

import pytest

from lora_moe_gb300 import binding as B
from lora_moe_gb300 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build folder of its own, and a stand-in for the compilers: nvcc writes its output, g++ fails."""
    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libmoe_lora.so"))
    monkeypatch.setattr(build, "FASTCALL", str(tmp_path / "fastcall.so"))
    monkeypatch.setattr(build, "_has_python_headers", lambda: True)
    commands = []

    def run(cmd, **kw):
        commands.append(os.path.basename(cmd[0]))
        if commands[-1] == "g++":
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no such header")
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(subprocess, "run", run)
    return commands


def test_the_library_is_built_without_it(tree):
    with pytest.warns(UserWarning, match="no such header"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.FASTCALL) and tree.count("g++") == 1
    build.build()                      # known not to build: not tried again
    assert tree.count("g++") == 1


def test_torch_that_does_not_import(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.warns(UserWarning, match="torch"):
        build.build()
    assert os.path.exists(build.LIB) and "g++" not in tree


def test_built_when_the_library_is_current(tree, monkeypatch):
    made = []

    def make():
        made.append(build.FASTCALL)
        with open(build.FASTCALL, "w"):
            pass
    monkeypatch.setattr(build, "_build_fastcall", make)
    build.build()
    compiled = len(tree)
    os.remove(build.FASTCALL)          # missing
    build.build()
    assert len(made) == 2
    os.utime(build.FASTCALL, (1, 1))   # older than its sources
    build.build()
    assert len(made) == 3
    build.build()
    assert len(made) == 3 and len(tree) == compiled


def test_name_says_what_it_was_built_against():
    import sysconfig
    import torch
    name = os.path.basename(build.FASTCALL)
    assert sysconfig.get_config_var("SOABI") in name and torch.__version__.split("+")[0] in name


def test_one_that_does_not_load(tmp_path, monkeypatch):
    B.lib()                            # (built, and not with the file below in its place)
    path = tmp_path / "fastcall.so"
    path.write_bytes(b"not a library")
    monkeypatch.setattr(build, "FASTCALL", str(path))
    monkeypatch.setattr(B, "_fast", None)
    with pytest.warns(UserWarning, match="ctypes"):
        assert B._load_fast() is B._NoFast
    assert B._load_fast() is B._NoFast
