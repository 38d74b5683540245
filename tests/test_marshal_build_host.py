"""The binding's native module is compiled against the installed PyTorch and
Python, and one made for another of them is not taken for it."""

import os
import subprocess

import pytest
import torch

from gqa_decode_attention_place_gb300 import _build


@pytest.fixture()
def compiler(monkeypatch, tmp_path):
    """A compiler that only notes what it was to write."""
    made = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write("module")
        made.append(out)
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(_build, "LIBDIR", str(tmp_path))
    monkeypatch.setattr(_build, "MARSHAL_PATH", str(tmp_path / "_gqa_marshal.so"), raising=False)
    monkeypatch.setattr(_build.subprocess, "run", run)
    return made


def test_made_once(compiler):
    first = _build.build_marshal()
    assert os.path.exists(first) and _build.build_marshal() == first and len(compiler) == 1
    _build.build_marshal(force=True)
    assert len(compiler) == 2


def test_another_pytorch_has_its_own(compiler, monkeypatch):
    first = _build.build_marshal()
    monkeypatch.setattr(torch, "__version__", "0.1.2+other")
    second = _build.build_marshal()
    assert second != first and len(compiler) == 2


def test_another_python_has_its_own(compiler, monkeypatch):
    first = _build.build_marshal()
    real = _build.sysconfig.get_config_var
    monkeypatch.setattr(_build.sysconfig, "get_config_var",
                        lambda name: "cpython-399-other" if name == "SOABI" else real(name))
    second = _build.build_marshal()
    assert second != first and len(compiler) == 2
