"""The build: the extension module is optional, the libraries are not. (The tree is built: nothing is compiled here.)"""
import os
import sys
import sysconfig

import pytest
import torch

import adamw_hybrid_optimizer_muon_b200 as ma
from adamw_hybrid_optimizer_muon_b200 import build as b


def no_torch(monkeypatch, tmp_path):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError


def no_compiler(monkeypatch, tmp_path):
    monkeypatch.setenv("CXX", str(tmp_path / "not-there"))


def failing_compiler(monkeypatch, tmp_path):
    monkeypatch.setenv("CXX", "false")


@pytest.mark.parametrize("broken", [no_torch, no_compiler, failing_compiler])
def test_the_libraries_are_built_without_the_extension_module(monkeypatch, tmp_path, capfd, broken):
    module = tmp_path / "_marshal.so"
    monkeypatch.setattr(b, "_marshal_path", lambda torch: str(module))  # not there yet
    broken(monkeypatch, tmp_path)
    assert b.build() == b.LIB
    assert os.path.exists(b.LIB)
    assert "marshal" in capfd.readouterr().err  # it says so
    assert not module.exists()


def test_the_extension_module_belongs_to_one_python_and_one_torch(monkeypatch):
    # what was built for another is not found: it reads the layout of that torch's tensors
    class Other:
        __version__ = "1.0.0"

    here = ma._marshal_path(torch)
    assert os.path.exists(here) and ma._marshal().__file__ == here
    assert not os.path.exists(ma._marshal_path(Other))
    monkeypatch.setattr(ma, "_TORCH", Other)
    monkeypatch.setattr(ma, "_MARSHAL", None)
    assert ma._marshal() is ma._Methods
    monkeypatch.setattr(ma, "_TORCH", torch)
    monkeypatch.setattr(ma, "_MARSHAL", None)
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-x86_64-linux-gnu")
    assert ma._marshal_path(torch) != here
    assert ma._marshal() is ma._Methods
