"""When the binding's compiled helper is made anew, and what build() does where
it cannot be made. The compiler is a stand-in that writes the output file."""
import os
import subprocess
import sysconfig

import pytest

from fp8_fine_grained_gb300 import build as libbuild


class Compiler:
    def __init__(self, rc=0):
        self.calls, self.rc = 0, rc

    def __call__(self, cmd, **kw):
        self.calls += 1
        if self.rc == 0:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("x")
        return subprocess.CompletedProcess(cmd, self.rc, "", "fatal error: Python.h: No such file or directory")


@pytest.fixture
def cc(monkeypatch, tmp_path):
    c = Compiler()
    monkeypatch.setattr(libbuild.subprocess, "run", c)
    monkeypatch.setattr(libbuild, "HELPER", str(tmp_path / "_tensors.so"))
    monkeypatch.setattr(libbuild, "BUILD", str(tmp_path / "_build"))
    return c


def test_made_once(cc):
    for _ in range(3):
        assert libbuild.build_helper() == libbuild.HELPER
    assert cc.calls == 1
    libbuild.build_helper(force=True)
    assert cc.calls == 2


def test_another_python(cc, monkeypatch):
    libbuild.build_helper()
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-x86_64-linux-gnu")
    libbuild.build_helper()
    libbuild.build_helper()
    assert cc.calls == 2


def test_another_torch(cc, monkeypatch, tmp_path):
    libbuild.build_helper()

    class Spec:
        submodule_search_locations = [str(tmp_path / "torch")]
    os.makedirs(tmp_path / "torch")
    monkeypatch.setattr(libbuild.importlib.util, "find_spec", lambda name: Spec)
    for version, calls in (("1", 2), ("1", 2), ("2", 3), ("2", 3)):
        (tmp_path / "torch" / "version.py").write_text("__version__ = '%s'\n" % version)
        libbuild.build_helper()
        assert cc.calls == calls


def test_newer_sources_and_a_helper_of_unknown_origin(cc):
    libbuild.build_helper()
    os.utime(libbuild.HELPER, (1, 1))
    libbuild.build_helper()
    assert cc.calls == 2
    os.remove(os.path.join(libbuild.BUILD, "tensors.made_for"))
    libbuild.build_helper()
    assert cc.calls == 3


def test_a_helper_that_cannot_be_made_leaves_the_library(cc, monkeypatch):
    cc.rc = 1
    monkeypatch.setattr(libbuild, "build_lib", lambda *a: "the library")
    with pytest.raises(RuntimeError, match="Python.h"):
        libbuild.build_helper()
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert libbuild.build() == "the library"
    with pytest.raises(RuntimeError, match="Python.h"):
        libbuild.build(strict=True)


def test_without_torch_or_a_compiler(cc, monkeypatch):
    monkeypatch.setattr(libbuild, "build_lib", lambda *a: "the library")

    def missing(cmd, **kw):
        raise FileNotFoundError(cmd[0])
    monkeypatch.setattr(libbuild.subprocess, "run", missing)
    with pytest.warns(RuntimeWarning, match="compiler"):
        assert libbuild.build() == "the library"
    monkeypatch.setattr(libbuild.importlib.util, "find_spec", lambda name: None)
    with pytest.warns(RuntimeWarning, match="torch is not installed"):
        assert libbuild.build() == "the library"


def test_the_library_alone_answers_without_the_helper(monkeypatch):
    """The older entry points need no helper; the others say what is missing."""
    import fp8_fine_grained_gb300 as fg
    libbuild.build_lib()
    monkeypatch.setattr(fg, "_helper", None)
    monkeypatch.setitem(__import__("sys").modules, "fp8_fine_grained_gb300._tensors", None)
    monkeypatch.delattr(fg, "_tensors", raising=False)
    assert fg.lib().fp8fg_version() > 0
    with pytest.raises(RuntimeError, match="_tensors.so is not built"):
        fg.grad_clip([], 1.0)
