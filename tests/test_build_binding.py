"""What building the extension module that checks tensors needs."""

import sys

import pytest

from fp8_quantized_skinny_amd import build


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """The commands of a build, none of them run."""
    seen = []
    monkeypatch.setattr(build, "_run", lambda cmd, verbose: seen.append(cmd) or "")
    monkeypatch.setattr(build.os, "replace", lambda a, b: None)
    return seen


def test_without_torch_the_library_alone_is_built(commands, monkeypatch):
    """Packing and quantizing need no torch, and nothing can call the extension module without it."""
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB
    assert len(commands) == len(build.SOURCES) + 1
    with pytest.raises(ImportError):
        build.build_binding()


def test_one_compiler_builds_everything(commands):
    assert build.build() == build.LIB
    assert len(commands) == len(build.SOURCES) + 2
    assert {cmd[0] for cmd in commands} == {build.hipcc()}
