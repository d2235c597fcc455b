"""When build() compiles what: the library for its sources and headers, the extension module for
its own source, the headers and the library.  The compilers are stand-ins that write empty files."""
import os
import sysconfig

import pytest

from lora_moe_expert_gb300 import build as b


class Tree:
    """A package folder of its own, with a clock: each write is a second after the one before."""

    def __init__(self, root, monkeypatch):
        self.now, self.runs, self.fail = 1_000_000_000, [], None
        self.pkg, self.include = str(root / "pkg"), str(root / "include")
        csrc = os.path.join(self.pkg, "csrc")
        os.makedirs(csrc)
        os.makedirs(self.include)
        for name in (*b.SOURCES, "mlg_py.cpp", "mlg_ptx.cuh"):
            self.write(os.path.join(csrc, name))
        for name in ("mlg.h", "mlg_test.h"):
            self.write(os.path.join(self.include, name))
        for name, at in (("PKG", self.pkg), ("CSRC", csrc), ("INCLUDE", self.include),
                         ("BUILD", os.path.join(self.pkg, "_build")),
                         ("LIBRARY", os.path.join(self.pkg, "libmlg.so")),
                         ("PY_MODULE", os.path.join(self.pkg, os.path.basename(b.PY_MODULE)))):
            monkeypatch.setattr(b, name, at)
        self.headers(root, monkeypatch, True)
        monkeypatch.setattr(b.subprocess, "run", self.compile)

    def headers(self, root, monkeypatch, there):
        at = root / f"python_{there}"
        os.makedirs(at, exist_ok=True)
        if there:
            (at / "Python.h").write_text("")
        paths = {**sysconfig.get_paths(), "include": str(at)}
        monkeypatch.setattr(b.sysconfig, "get_paths", lambda: paths)

    def write(self, path):
        with open(path, "w"):
            pass
        self.now += 1
        os.utime(path, (self.now, self.now))

    def compile(self, cmd, check):
        out = cmd[cmd.index("-o") + 1]
        what = "module" if cmd[0] == "g++" else "library" if "-shared" in cmd else "unit"
        self.runs.append(what)
        if self.fail == what:
            raise b.subprocess.CalledProcessError(1, cmd)
        self.write(out)

    def built(self):
        """What a build() compiles now."""
        self.runs.clear()
        b.build()
        return set(self.runs)


@pytest.fixture
def tree(tmp_path, monkeypatch):
    return Tree(tmp_path, monkeypatch)


ALL = {"unit", "library", "module"}


def test_builds_once(tree):
    assert tree.built() == ALL
    assert tree.built() == set()


@pytest.mark.parametrize("name", ["csrc/mlg_rows.cu", "csrc/mlg_ptx.cuh", "../include/mlg.h",
                                  "../include/mlg_test.h"])
def test_a_source_of_the_library(tree, name):
    tree.built()
    tree.write(os.path.join(tree.pkg, name))
    assert tree.built() == ALL
    assert tree.built() == set()


def test_the_modules_own_source(tree):
    tree.built()
    tree.write(os.path.join(tree.pkg, "csrc", "mlg_py.cpp"))
    assert tree.built() == {"module"}
    assert tree.built() == set()


def test_without_pythons_headers(tree, tmp_path, monkeypatch):
    tree.headers(tmp_path, monkeypatch, False)
    assert tree.built() == {"unit", "library"}
    assert tree.built() == set()


def test_a_failed_module_leaves_none_and_is_built_again(tree):
    """An old module with a new library would marshal the old calls."""
    tree.built()
    tree.write(os.path.join(tree.include, "mlg.h"))
    tree.fail = "module"
    with pytest.raises(b.subprocess.CalledProcessError):
        b.build()
    assert not os.path.exists(b.PY_MODULE)
    tree.fail = None
    assert tree.built() == {"module"}
    assert tree.built() == set()


def test_a_module_of_another_interpreter_is_not_loaded():
    assert os.path.basename(b.PY_MODULE) == "_mlg_py" + sysconfig.get_config_var("EXT_SUFFIX")


def test_an_untagged_module_is_removed(tree):
    """Any interpreter would load it."""
    old = os.path.join(tree.pkg, "_mlg_py.so")
    tree.write(old)
    tree.built()
    assert not os.path.exists(old)
