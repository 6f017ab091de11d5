"""The native front of the hard selections' Python side when its file is of another time (no GPU)."""
import os
import warnings

import pytest

pytest.importorskip("torch")
from sparse_selection_primitive_amd import hard


def bind(monkeypatch, path):
    for name in ("torch", "_raw_stream", "_current_device", "_native"):
        monkeypatch.setattr(hard, name, getattr(hard, name))  # put back afterwards
    hard._native = None
    monkeypatch.setattr(hard, "_NATIVE_PATH", str(path))
    hard._bind()
    return hard._native


def test_a_front_without_some_of_the_calls_is_named(monkeypatch, tmp_path):
    old = tmp_path / "_binding.py"
    calls = [n for n in hard._NATIVE_CALLS if n != "beam_select"]
    old.write_text("\n".join(f"def {n}(*a): raise AssertionError" for n in ["bind", "on_failure", *calls]))
    with pytest.warns(RuntimeWarning, match="out of date.*beam_select"):
        assert bind(monkeypatch, old) is None


def test_a_whole_front_is_used_and_no_file_is_none(monkeypatch, tmp_path):
    new = tmp_path / "_binding.py"
    new.write_text("bound = []\ndef bind(*a): bound.extend(a)\ndef on_failure(f): pass\n" +
                   "\n".join(f"def {n}(*a): pass" for n in hard._NATIVE_CALLS if not n.endswith("_bytes")))
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        front = bind(monkeypatch, new)
        assert front is not None and len(front.bound) == len(hard._NATIVE_CALLS)
        assert bind(monkeypatch, tmp_path / "none.so") is None
        if os.path.exists(os.path.join(os.path.dirname(hard.__file__), "_binding.so")):
            assert bind(monkeypatch, os.path.join(os.path.dirname(hard.__file__), "_binding.so")) is not None
