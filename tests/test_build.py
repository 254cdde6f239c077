"""The build's two products: the library, and the paged-cache calls' binding, which only those calls need."""
import os
import subprocess
import sys

import pytest
import torch

from post_activation_quantization_b200 import build


def _fail(*a, **k):
    raise subprocess.CalledProcessError(1, "g++")


def test_library_is_built_where_the_binding_cannot_be(monkeypatch, capsys):
    monkeypatch.setattr(build, "build_marshal", _fail)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert "no binding" in capsys.readouterr().err


def test_binding_belongs_to_this_python_and_torch(monkeypatch):
    build.build()
    path = build.marshal_path()
    assert os.path.exists(path)
    assert sys.implementation.cache_tag in os.path.basename(path) and torch.__version__ in os.path.basename(path)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert build.marshal_path() != path


def test_binding_of_an_older_source_does_not_outlive_a_failed_build(monkeypatch, tmp_path):
    old = tmp_path / "_marshal.so"
    old.write_bytes(b"")
    os.utime(old, (0, 0))
    monkeypatch.setattr(build, "marshal_path", lambda: str(old))
    monkeypatch.setattr(build.subprocess, "check_call", _fail)
    with pytest.raises(subprocess.CalledProcessError):
        build.build_marshal()
    assert not old.exists()
