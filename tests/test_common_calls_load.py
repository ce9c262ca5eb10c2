"""The optional module of the common calls is never a condition of loading the library."""
import pytest

import int8_quantized_gemm_gb300 as q8
from int8_quantized_gemm_gb300 import build


@pytest.fixture
def unloaded(monkeypatch):
    """The package before its first call."""
    build.build()
    monkeypatch.setattr(q8, "_lib", None)
    monkeypatch.setattr(q8, "_calls", None)


def at(monkeypatch, path):
    monkeypatch.setattr(build, "calls_path", lambda: str(path))


def test_no_module(unloaded, monkeypatch, tmp_path):
    at(monkeypatch, tmp_path / "none.so")
    assert q8.load() is q8._lib and q8._calls is None


@pytest.mark.parametrize("content", [b"", b"no shared object"])
def test_a_broken_module_is_reported_and_not_used(unloaded, monkeypatch, tmp_path, content):
    path = tmp_path / "broken.so"
    path.write_bytes(content)
    at(monkeypatch, path)
    with pytest.warns(RuntimeWarning, match="the binding makes its calls itself"):
        lib = q8.load()
    assert lib is q8._lib and q8._calls is None
    assert q8.status_string(q8.Q8_OK)               # the library's calls work
    assert q8.load() is lib


def test_a_library_of_another_kind_is_reported_and_not_used(unloaded, monkeypatch):
    """A shared object that is no module of Python's: it loads, but has no entry for the interpreter."""
    at(monkeypatch, build.LIB)
    with pytest.warns(RuntimeWarning, match="the binding makes its calls itself"):
        q8.load()
    assert q8._calls is None
