"""Building the library and the optional module of the common calls, with stand-ins for the compilers: no GPU, nothing compiled."""
import os

import pytest

from int8_quantized_gemm_gb300 import build

WORKS = """#!/bin/sh
while [ $# -gt 0 ]; do
    if [ "$1" = "-o" ]; then echo "$STAND_IN" > "$2"; fi
    shift
done
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """An empty place for what is built, and compilers that write $STAND_IN to their output."""
    tool = tmp_path / "compiler"
    tool.write_text(WORKS)
    tool.chmod(0o755)
    out = tmp_path / "_lib"
    monkeypatch.setattr(build, "OUT_DIR", str(out))
    monkeypatch.setattr(build, "LIB", str(out / "libq8.so"))
    monkeypatch.setenv("NVCC", str(tool))
    monkeypatch.setenv("CXX", str(tool))
    monkeypatch.setenv("STAND_IN", "first")
    return out


def content(path):
    with open(path) as f:
        return f.read().strip()


def test_both_are_built(tree):
    assert build._stale()
    assert build.build() == build.LIB and content(build.LIB) == "first" and content(build.calls_path()) == "first"
    assert not build._stale()
    assert sorted(os.listdir(tree)) == sorted([os.path.basename(build.LIB), os.path.basename(build.calls_path())])


@pytest.mark.parametrize("compiler", ["/bin/false", "/nonexistent/compiler"])
def test_a_module_that_does_not_compile_leaves_no_older_one(tree, monkeypatch, capsys, compiler):
    """An older module would make calls of the older library's form to the new one."""
    build.build()
    other = tree / "_q8_calls_cpython_39_torch_2_0_0.so"      # of another interpreter, for the older library
    other.write_text("first")
    monkeypatch.setenv("STAND_IN", "second")
    monkeypatch.setenv("CXX", compiler)
    build.build(force=True)
    assert content(build.LIB) == "second"
    assert not os.path.exists(build.calls_path()) and not other.exists()
    assert "the binding makes these calls itself" in capsys.readouterr().err
    assert not build._stale()                                # it is not tried again at every build

    monkeypatch.setenv("STAND_IN", "third")
    monkeypatch.setenv("CXX", os.environ["NVCC"])
    build.build(force=True)
    assert content(build.LIB) == content(build.calls_path()) == "third"
    assert not os.path.exists(build.calls_path() + ".none") and not build._stale()


def test_a_library_that_does_not_compile_changes_nothing(tree, monkeypatch):
    """The older library keeps the module that was built with it."""
    build.build()
    monkeypatch.setenv("STAND_IN", "second")
    monkeypatch.setenv("NVCC", "/bin/false")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build(force=True)
    assert content(build.LIB) == content(build.calls_path()) == "first"
