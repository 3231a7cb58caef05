"""The extension module that checks tensors is taken only by the torch that it was built for."""

import pytest
import torch

from fp8_quantized_skinny_amd import _lib


def test_a_binding_of_another_torch_is_refused(monkeypatch):
    assert _lib.native() is not None
    monkeypatch.setattr(_lib, "_NATIVE", None)
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    with pytest.raises(ImportError, match="0.0.0"):
        _lib.native()
    monkeypatch.undo()
    assert _lib.native().torch_version == torch.__version__
