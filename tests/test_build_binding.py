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
