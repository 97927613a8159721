"""The build: the extension module is optional, the libraries are not. (The tree is built: nothing is compiled here.)"""
import os
import sys

import pytest

from adamw_hybrid_optimizer_muon_b200 import build as b


def no_torch(monkeypatch, tmp_path):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError


def no_compiler(monkeypatch, tmp_path):
    monkeypatch.setenv("CXX", str(tmp_path / "not-there"))


def failing_compiler(monkeypatch, tmp_path):
    monkeypatch.setenv("CXX", "false")


@pytest.mark.parametrize("broken", [no_torch, no_compiler, failing_compiler])
def test_the_libraries_are_built_without_the_extension_module(monkeypatch, tmp_path, capfd, broken):
    monkeypatch.setattr(b, "MARSHAL", str(tmp_path / "_marshal.so"))  # not there yet
    broken(monkeypatch, tmp_path)
    assert b.build() == b.LIB
    assert os.path.exists(b.LIB)
    assert "marshal" in capfd.readouterr().err  # it says so
    assert not os.path.exists(b.MARSHAL)
