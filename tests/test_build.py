"""The build on hosts without PyTorch, and the binding of another PyTorch."""
import json
import os
import sys

import pytest

from depth_weighted_scatter_gb300 import _build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A built library, and a binding and its key of the test's own."""
    _build.build()
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_token_ops.so"))
    monkeypatch.setattr(_build, "BINDING_KEY", str(tmp_path / "binding.json"))
    return tmp_path


def test_library_without_pytorch(elsewhere, monkeypatch, capsys):
    """The C library needs no PyTorch, no headers of it, and none of Python."""
    monkeypatch.setitem(sys.modules, "torch", None)
    assert _build.build() == _build.LIB and os.path.exists(_build.LIB)
    assert not os.path.exists(_build.BINDING) and "PyTorch" in capsys.readouterr().err


def test_library_without_headers(elsewhere, monkeypatch, capsys):
    monkeypatch.setattr(_build, "_torch_dir", lambda: str(elsewhere))
    assert _build.build() == _build.LIB
    assert not os.path.exists(_build.BINDING) and "python_variable.h" in capsys.readouterr().err


def test_binding_of_another_pytorch_is_not_up_to_date(elsewhere):
    key = _build._binding_key()
    (elsewhere / "_token_ops.so").write_bytes(b"")
    assert not _build.binding_up_to_date()                  # nobody knows what it was made for
    (elsewhere / "binding.json").write_text(json.dumps(key))
    assert _build.binding_up_to_date()
    for name in key:
        (elsewhere / "binding.json").write_text(json.dumps({**key, name: "another"}))
        assert not _build.binding_up_to_date()
