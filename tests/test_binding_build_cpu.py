"""The extension module _moe_torch.so: when it is built again, and what an import
says without it."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

import __graft_entry__

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def build(monkeypatch, tmp_path):
    b = __graft_entry__._build_module()
    if b.stale(b.OUT):
        b.build()
    for name in ("OUT", "BINDING_OUT"):
        at = tmp_path / os.path.basename(getattr(b, name))
        shutil.copyfile(getattr(b, name), at)
        monkeypatch.setattr(b, name, str(at))
    assert not b.stale(b.OUT) and not b.stale(b.BINDING_OUT)
    return b


def test_torch_version_is_torchs(build):
    assert build.torch_version() == torch.__version__


def test_a_missing_module_is_stale(build):
    os.remove(build.BINDING_OUT)
    assert build.stale(build.BINDING_OUT) and build.stale(build.OUT)


def test_a_module_older_than_its_source_is_stale(build):
    os.utime(build.BINDING_OUT, (1, 1))
    assert build.stale(build.BINDING_OUT) and build.stale(build.OUT)


def test_a_module_built_with_another_torch_is_stale(build, monkeypatch):
    monkeypatch.setattr(build, "torch_version", lambda: torch.__version__ + ".1")
    assert build.stale(build.BINDING_OUT) and build.stale(build.OUT)
    monkeypatch.setattr(build, "torch_version", lambda: torch.__version__[:-1])
    assert build.stale(build.BINDING_OUT) and build.stale(build.OUT)


def imported(tmp_path, change):
    """The error of importing a copy of the package, after `change` of its module."""
    b = __graft_entry__._build_module()
    if b.stale(b.OUT):
        b.build()
    at = tmp_path / "sparse_expert_gemv_gb300"
    shutil.copytree(b.HERE, at, ignore=shutil.ignore_patterns("csrc", "__pycache__", "*timeline*"))
    change(at / "_moe_torch.so")
    r = subprocess.run([sys.executable, "-c", "import sparse_expert_gemv_gb300"], cwd=tmp_path,
                       capture_output=True, text=True, env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode != 0
    return r.stderr


def test_import_without_the_module(tmp_path):
    err = imported(tmp_path, os.remove)
    assert "_moe_torch.so is missing or does not load" in err and "g.build()" in err


def test_import_of_a_module_of_another_torch(tmp_path):
    def relabel(so):
        data, at = so.read_bytes(), f"built with torch {torch.__version__}".encode()
        assert data.count(at + b"\0") >= 1
        so.write_bytes(data.replace(at, at[:-1] + b"~"))
    err = imported(tmp_path, relabel)
    assert f"this is torch {torch.__version__}" in err and "g.build()" in err
