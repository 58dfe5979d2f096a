"""The compiled binding follows the Python and torch that it was built for (CPU)."""

import pytest

import exact_memory_efficient_b200 as m
from exact_memory_efficient_b200 import build as b


@pytest.fixture(scope="module", autouse=True)
def built():
    b.build()


def test_a_binding_of_another_torch_or_python_is_stale(monkeypatch):
    assert not b.needs_binding()
    monkeypatch.setattr("torch.__version__", "0.0.0+other")
    assert b.needs_binding()
    monkeypatch.undo()
    assert not b.needs_binding()
    real = b.sysconfig.get_config_var
    monkeypatch.setattr(b.sysconfig, "get_config_var", lambda k: "cpython-00-other" if k == "SOABI" else real(k))
    assert b.needs_binding()


def test_a_stale_binding_is_not_loaded(monkeypatch):
    """The message names the command, which then does build it."""
    monkeypatch.setattr(m, "_BINDING", None)
    monkeypatch.setattr("torch.__version__", "0.0.0+other")
    with pytest.raises(RuntimeError, match="exact_memory_efficient_b200.build"):
        m.load_binding()


def test_a_rebuilt_binding_fits(monkeypatch, tmp_path):
    monkeypatch.setattr(b, "BINDING_PATH", str(tmp_path / "_binding.so"))
    assert b.needs_binding()
    b.build_binding()
    assert not b.needs_binding()


def without_python_headers(monkeypatch, tmp_path):
    monkeypatch.setattr(b, "BINDING_PATH", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(b.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})


def test_the_library_is_built_where_the_binding_cannot_be(monkeypatch, tmp_path, capfd):
    """The C library needs nvcc alone; what the binding lacks is said, and load_binding() still fails loudly."""
    without_python_headers(monkeypatch, tmp_path)
    assert b.build() == b.LIB_PATH
    said = capfd.readouterr().err
    assert "_binding.so" in said and "Python.h" in said
    with pytest.raises(RuntimeError, match="Python.h"):
        b.build_binding()
    monkeypatch.setattr(m, "_BINDING", None)
    with pytest.raises(RuntimeError, match="there is no fallback"):
        m.load_binding()


def test_each_thing_that_the_binding_needs(monkeypatch):
    assert b.binding_lacks() == []
    monkeypatch.setattr(b.shutil, "which", lambda name: None if name == "g++" else "/usr/bin/" + name)
    assert b.binding_lacks() == ["g++"]
    monkeypatch.undo()
    monkeypatch.setitem(__import__("sys").modules, "torch", None)      # import torch raises ImportError
    assert b.binding_lacks() == ["torch"]
