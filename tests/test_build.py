"""How the library and the compiled part of the Python binding are built, on a tree of two small sources (no GPU needed)."""
import ctypes
import importlib
import os
import subprocess

import pytest

b = importlib.import_module("medusa_tree_speculative_verify_gb300.build")

CALLS = """#include <Python.h>
static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, nullptr, nullptr, nullptr, nullptr, nullptr};
PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A package of one kernel source and one of the binding, under the module's own rules; and the commands that are run."""
    pkg = tmp_path / "pkg"
    (pkg / "csrc").mkdir(parents=True)
    (pkg / "csrc" / "one.cu").write_text('extern "C" int answer() { return 42; }\n')
    (pkg / "csrc" / "calls.cpp").write_text(CALLS)
    for name, path in (("PKG", pkg), ("CSRC", pkg / "csrc"), ("BUILD", pkg / "_build"), ("LIB", pkg / "libmedusa_verify.so"),
                       ("CALLS_SRC", pkg / "csrc" / "calls.cpp"), ("CALLS", pkg / "_calls.so")):
        monkeypatch.setattr(b, name, str(path), raising=False)
    commands, run = [], subprocess.run

    def spy(cmd, *args, **kw):
        commands.append([os.path.basename(x) for x in cmd])
        return run(cmd, *args, **kw)

    monkeypatch.setattr(b.subprocess, "run", spy)
    return pkg, commands


def bindings(pkg):
    return sorted(p for p in os.listdir(pkg) if p.startswith("_calls") and p.endswith(".so"))


def no_torch(monkeypatch):
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name, *args: None)


def test_library_needs_no_torch(tree, monkeypatch):
    pkg, _ = tree
    no_torch(monkeypatch)
    assert ctypes.CDLL(b.build()).answer() == 42
    assert not bindings(pkg)
    with pytest.raises(RuntimeError, match="torch"):
        b.build_calls()
    b.build()                                                 # as often as it is asked for


def test_binding_that_does_not_compile_leaves_the_library(tree):
    pkg, _ = tree
    (pkg / "csrc" / "calls.cpp").write_text("#error no such binding\n")
    with pytest.raises(RuntimeError):
        b.build()
    assert ctypes.CDLL(b.LIB).answer() == 42 and not bindings(pkg)
    (pkg / "csrc" / "calls.cpp").write_text(CALLS)
    b.build()
    assert len(bindings(pkg)) == 1


def test_each_is_rebuilt_for_its_own_sources(tree):
    pkg, commands = tree
    b.build()
    made = bindings(pkg)
    assert len(made) == 1 and any("one.cu" in c for c in commands)
    commands.clear()
    b.build()
    assert not commands                                       # nothing is out of date
    os.remove(pkg / made[0])
    b.build()
    assert bindings(pkg) == made and not any("one.cu" in c for c in commands)
    commands.clear()
    later = os.path.getmtime(pkg / made[0]) + 10
    os.utime(pkg / "csrc" / "one.cu", (later, later))
    b.build()
    assert any("one.cu" in c for c in commands) and not any("calls.cpp" in c for c in commands)
