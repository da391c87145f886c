"""The extension that calls torch's C++ interface belongs to one torch version: another one's is rebuilt, and never loaded."""
import pytest
import torch

import ragged_variable_length_b200 as rv
from ragged_variable_length_b200 import build as rbuild


def test_current_extension_names_its_torch():
    path = rbuild.build_torchcall()
    assert rbuild.torchcall_is_current(path)
    assert rv._load_torchcall().built_for == torch.__version__


def test_extension_of_another_torch_is_rebuilt(monkeypatch):
    path = rbuild.build_torchcall()
    runs = []
    monkeypatch.setattr(rbuild.subprocess, "run", lambda cmd, **kw: runs.append(cmd))
    monkeypatch.setattr(rbuild.os, "replace", lambda a, b: None)
    assert rbuild.build_torchcall() == path and not runs
    monkeypatch.setattr(torch, "__version__", "2.10.0")
    assert not rbuild.torchcall_is_current(path)
    rbuild.build_torchcall()
    assert len(runs) == 1 and '-DRAGGED_TORCH_VERSION="2.10.0"' in runs[0]


def test_extension_of_another_torch_is_not_loaded(monkeypatch):
    rbuild.build_torchcall()
    monkeypatch.setattr(rv, "_tc", None)
    monkeypatch.setattr(torch, "__version__", "2.10.0")
    with pytest.raises(RuntimeError, match="another torch"):
        rv._load_torchcall()


def test_missing_extension_is_not_current(tmp_path):
    assert not rbuild.torchcall_is_current(str(tmp_path / "none.so"))
