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


def test_binding_belongs_to_one_torch_and_interpreter(tree, monkeypatch, tmp_path):
    """Another torch, or another version in its place, or another interpreter: what was built for the old one is not taken."""
    pkg, _ = tree
    b.build()
    assert not b._stale()
    other = tmp_path / "torch"
    other.mkdir()
    monkeypatch.setattr(b, "torch_dir", lambda: str(other))
    (other / "version.py").write_text("__version__ = '2.0.0'\n")
    assert b._stale()


def test_binding_follows_torchs_version_and_the_interpreters(tree, monkeypatch, tmp_path):
    pkg, _ = tree
    fake = tmp_path / "torch"
    fake.mkdir()
    (fake / "version.py").write_text("__version__ = '2.0.0'\n")
    monkeypatch.setattr(b, "torch_dir", lambda: str(fake))
    names = {b.calls_path()}
    (fake / "version.py").write_text("__version__ = '2.0.1'\n")
    names.add(b.calls_path())
    monkeypatch.setattr(b.sys, "version", b.sys.version + " (other)")
    names.add(b.calls_path())
    monkeypatch.setattr(b.sysconfig, "get_config_var", lambda name: ".cpython-399-x.so")
    names.add(b.calls_path())
    assert len(names) == 4 and all(os.path.basename(n).startswith("_calls") for n in names)


def test_binding_of_another_name_is_not_loaded():
    """What is imported is the file that belongs to this torch and interpreter."""
    code = ("import medusa_tree_speculative_verify_gb300 as mv, importlib;"
            "print(mv._load_calls().__file__ == importlib.import_module(mv.__name__ + '.build').calls_path())")
    r = subprocess.run([b.sys.executable, "-c", code], capture_output=True, text=True, cwd=b.ROOT)
    assert r.stdout.strip() == "True", r.stdout + r.stderr
