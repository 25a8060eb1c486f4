"""The marshalling extension belongs to the torch and the Python it was compiled for."""

import subprocess
import sysconfig

import pytest
import torch

from block_sparse_gqa_03_b200 import build as msa_build
from block_sparse_gqa_03_b200 import msa


def test_its_name_holds_both_versions():
    msa_build.build()
    path = msa_build.marshal_path()
    assert path == msa.MARSHAL_PATH
    assert torch.__version__ in path and path.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    msa._marshal_module()


@pytest.mark.parametrize("what", ["torch", "python"])
def test_one_of_another_version_is_neither_current_nor_loaded(what, monkeypatch):
    msa_build.build()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "9.9.9")
    else:
        monkeypatch.setattr(sysconfig, "get_config_var", lambda name: ".cpython-999.so")
    commands = []
    monkeypatch.setattr(subprocess, "run", lambda cmd, check: commands.append(cmd))
    monkeypatch.setattr(msa_build.os, "replace", lambda a, b: None)
    assert msa_build.build_marshal() == msa_build.marshal_path() != msa.MARSHAL_PATH
    assert len(commands) == 1  # compiled anew, although the sources are no newer
    assert any(c.startswith("-D_GLIBCXX_USE_CXX11_ABI=") for c in commands[0])
    monkeypatch.setattr(msa, "MARSHAL_PATH", msa_build.marshal_path())
    with pytest.raises(RuntimeError, match="not built"):
        msa._marshal_module()


def test_the_library_builds_without_python_headers(monkeypatch, tmp_path, capsys):
    msa_build.build()
    monkeypatch.setattr(torch, "__version__", "9.9.9")  # none is built for it
    monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert msa_build.build() == msa_build.LIB
    assert "Python.h" in capsys.readouterr().err
