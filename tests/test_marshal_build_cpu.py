"""The compiled argument marshalling belongs to one PyTorch and one Python: it
is rebuilt for others, and a file that does not load is not passed over in
silence."""
import os
import sys

import pytest
import torch

import tensor_matmul_collective_gb300 as pkg
from tensor_matmul_collective_gb300 import build, coc


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_another_pytorch_makes_it_stale(monkeypatch):
    assert not build._marshal_stale()
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    assert build._marshal_stale()


def test_another_python_makes_it_stale(monkeypatch):
    monkeypatch.setattr(sys, "version", "0")
    assert build._marshal_stale()


def test_without_a_record_it_is_stale(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "MARSHAL_FOR", os.fspath(tmp_path / "none"))
    assert build._marshal_stale()


def test_a_file_that_does_not_load_is_reported(monkeypatch):
    monkeypatch.setattr(coc, "_native", None)
    monkeypatch.setitem(sys.modules, "tensor_matmul_collective_gb300._coc_marshal", None)     # import raises ImportError
    monkeypatch.delattr(pkg, "_coc_marshal", raising=False)
    with pytest.warns(RuntimeWarning, match="_coc_marshal"):
        assert coc._marshal() is False
    assert coc._marshal() is False


def test_it_loads():
    assert coc._marshal()
