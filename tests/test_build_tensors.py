"""The native part of the Python binding belongs to one Python and one torch (no GPU needed)."""
import os

import pytest
import torch

from recurrent_cell_unroll_gb300 import _build, binding


def test_another_torch_does_not_load_it(monkeypatch):
    _build.build()
    path = _build.tensors_path()
    assert os.path.exists(path) and torch.__version__ in os.path.basename(path)
    monkeypatch.setattr(binding, "_tensors_module", None)
    assert binding._tensors().adamw_rows
    monkeypatch.setattr(binding, "_tensors_module", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    other = _build.tensors_path()
    assert other != path
    with pytest.raises(RuntimeError, match="not found"):
        binding._tensors()


def test_it_is_built_for_each_torch(monkeypatch):
    asked = []

    def command(out):
        asked.append(out)
        return ["touch", out]
    monkeypatch.setattr(torch, "__version__", "0.0.2")
    monkeypatch.setattr(_build, "_tensors_command", command)
    path = _build.tensors_path()
    try:
        _build.build()
        assert len(asked) == 1 and os.path.exists(path)
        _build.build()
        assert len(asked) == 1
    finally:
        if os.path.exists(path):
            os.remove(path)


@pytest.mark.parametrize("command", [["false"], ["no-such-compiler"]])
def test_without_it_the_library_is_built(monkeypatch, tmp_path, command):
    _build.build()
    lib = tmp_path / "librcu.so"
    monkeypatch.setattr(_build, "LIB", str(lib))
    monkeypatch.setattr(_build, "tensors_path", lambda: str(tmp_path / "tensors.so"))
    monkeypatch.setattr(_build, "_tensors_command", lambda out: command)
    with pytest.raises(RuntimeError, match="native part"):
        _build.build()
    assert lib.exists()
