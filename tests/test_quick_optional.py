"""The plain calls' faster way is built for one interpreter and one torch, and the library does without it (CPU)."""
import os
import warnings

import pytest

import kda_state_gb300.binding as binding
from kda_state_gb300 import _build


@pytest.fixture
def apart(tmp_path, monkeypatch):
    """A place of its own for the module and its key, beside the library that is built."""
    _build.build()
    monkeypatch.setattr(_build, "QUICK", str(tmp_path / "_quick.so"))
    monkeypatch.setattr(_build, "QUICK_KEY", str(tmp_path / "_quick.key"))
    monkeypatch.setattr(binding, "QUICK_PATH", str(tmp_path / "_quick.so"))
    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "_quick", None)
    return tmp_path


def loads(path, key):
    """Whether lib() takes the module at path, which warns where it does not."""
    (path / "_quick.key").write_text(key)
    with warnings.catch_warnings(record=True) as told:
        warnings.simplefilter("always")
        L = binding.lib()
    assert L.kda_status_string(0) and binding.lib() is L
    assert (binding._quick is None) == any("calls take longer" in str(w.message) for w in told)
    return binding._quick is not None


def test_the_library_loads_without_the_module(apart):
    assert not loads(apart, _build.quick_key())


def test_a_module_that_does_not_load_is_left(apart):
    (apart / "_quick.so").write_bytes(b"no shared object")
    assert not loads(apart, _build.quick_key())


def test_a_module_built_for_another_torch_is_not_loaded(apart, monkeypatch):
    (apart / "_quick.so").write_bytes(b"never opened")
    monkeypatch.setattr(binding.importlib.machinery, "ExtensionFileLoader", lambda *a: pytest.fail("it was opened"))
    assert not loads(apart, _build.quick_key().replace("torch ", "torch 0."))


def test_the_module_goes_by_what_it_was_built_for(apart, monkeypatch):
    built = []

    def compiled():
        built.append(1)
        path = str(apart / "new.tmp")
        with open(path, "w") as f:
            f.write("module %d" % len(built))
        return path
    monkeypatch.setattr(_build, "_compile_quick", compiled)
    lib_time = os.path.getmtime(_build.LIB)
    _build.build()
    _build.build()
    assert len(built) == 1 and _build.up_to_date()
    monkeypatch.setattr(_build, "quick_key", lambda: "another torch")
    assert not _build.up_to_date()
    _build.build()
    assert len(built) == 2 and _build.quick_built_for() == "another torch"
    os.remove(_build.QUICK)
    _build.build()
    assert len(built) == 3 and os.path.getmtime(_build.LIB) == lib_time


@pytest.mark.parametrize("fault", [RuntimeError("g++ failed"), FileNotFoundError("g++"), ImportError("torch")])
def test_a_build_that_fails_is_a_warning_and_is_not_tried_again(apart, monkeypatch, fault):
    tried = []

    def compiled():
        tried.append(1)
        raise fault
    monkeypatch.setattr(_build, "_compile_quick", compiled)
    with pytest.warns(RuntimeWarning, match="is not built"):
        assert _build.build() == _build.LIB
    assert _build.up_to_date() and _build.build() == _build.LIB and len(tried) == 1
    assert not loads(apart, _build.quick_built_for())


def test_without_torch_only_the_library_is_built(apart, monkeypatch):
    def absent():
        raise ImportError("No module named 'torch'")
    monkeypatch.setattr(_build, "quick_key", absent)
    assert _build.up_to_date() and _build.build() == _build.LIB and not os.path.exists(_build.QUICK)
