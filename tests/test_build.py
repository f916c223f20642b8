"""The build: the CUDA library depends on nvcc alone, the marshalling module is
optional.  Compilers are stood in for."""
import os
import subprocess
import sysconfig

import pytest

from fp8_relu_mlp_b200 import build as B


class Compilers:
    """Instead of subprocess.run: writes each output, fails on what it is told to."""

    def __init__(self):
        self.ran, self.fails = [], set()

    def __call__(self, cmd, **kw):
        self.ran.append(cmd)
        if any(f in cmd for f in self.fails):
            return subprocess.CompletedProcess(cmd, 1, "", "no such thing")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(" ".join(cmd))
        return subprocess.CompletedProcess(cmd, 0, "", "")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libfp8mlp.so"))
    monkeypatch.setattr(B, "MARSHAL", str(tmp_path / os.path.basename(B.MARSHAL)))
    monkeypatch.setattr(B, "UNTAGGED", str(tmp_path / "_marshal.so"))
    monkeypatch.setenv("CXX", "the-compiler")
    run = Compilers()
    monkeypatch.setattr(B.subprocess, "run", run)
    return run


def no_toolkit():
    raise RuntimeError("nvcc not found")


def test_both_are_built_once(tree):
    assert B.build() == B.LIB and os.path.exists(B.LIB) and os.path.exists(B.MARSHAL)
    n = len(tree.ran)
    assert B.build() == B.LIB and len(tree.ran) == n
    assert B.build(force=True) == B.LIB and len(tree.ran) == 2 * n


@pytest.mark.parametrize("how", ["fails", "is not there"])
def test_the_library_is_built_when_the_module_is_not(tree, monkeypatch, how):
    open(B.MARSHAL, "w").close()  # of other sources
    if how == "fails":
        tree.fails.add("the-compiler")
    else:
        def run(cmd, **kw):
            if cmd[0] == "the-compiler":
                raise FileNotFoundError(cmd[0])
            return tree(cmd, **kw)
        monkeypatch.setattr(B.subprocess, "run", run)
    with pytest.warns(UserWarning, match="stays in Python"):
        assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(B.MARSHAL)


def test_headers_of_another_torch(tree, monkeypatch):
    monkeypatch.setattr(B, "TORCH_HEADERS", B.TORCH_HEADERS + ("torch/no/such.h",))
    assert B.build() == B.LIB and B.build_marshal() is None
    assert all(c[0] != "the-compiler" for c in tree.ran)


def test_every_torch_header_of_the_module_is_asked_for():
    inc = [ln.split("<")[1].split(">")[0] for ln in open(os.path.join(B.CSRC, "binding.cpp")) if ln.startswith("#include <")]
    assert {h for h in inc if "/" in h} == set(B.TORCH_HEADERS)


def test_a_current_library_needs_no_toolkit(tree, monkeypatch):
    B.build()
    n = len(tree.ran)
    monkeypatch.setattr(B, "nvcc", no_toolkit)
    assert B.build() == B.LIB and os.path.exists(B.MARSHAL) and len(tree.ran) == n
    # nor without the module
    os.remove(B.MARSHAL)
    assert B.build() == B.LIB and len(tree.ran) == n
    # a library that is not current does
    os.remove(B.LIB)
    with pytest.raises(RuntimeError, match="nvcc"):
        B.build()


def test_the_library_failing_is_an_error(tree, monkeypatch):
    monkeypatch.setattr(B, "nvcc", lambda: "the-nvcc")
    tree.fails.add("the-nvcc")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        B.build()


def test_the_module_is_named_for_this_python(tree):
    assert os.path.basename(B.MARSHAL) == "_marshal" + sysconfig.get_config_var("EXT_SUFFIX")
    open(B.UNTAGGED, "w").close()
    B.build()
    assert not os.path.exists(B.UNTAGGED) and os.path.exists(B.MARSHAL)
