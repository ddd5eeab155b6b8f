"""The marshalling module's file: which one is loaded, and when it is built anew."""
import os
import sysconfig

import pytest
import torch

import fine_grained_moe_gemm_b200 as moe
from fine_grained_moe_gemm_b200 import build


def test_binding_file_names_torch_and_the_interpreter():
    """A second interpreter or torch in the same checkout must not find the other's module fresh and load it."""
    name = build.binding_path()
    suffix = sysconfig.get_config_var("EXT_SUFFIX")      # such as .cpython-312-x86_64-linux-gnu.so
    assert sysconfig.get_config_var("SOABI") in suffix and name.endswith(suffix)
    assert "".join(c if c.isalnum() else "_" for c in torch.__version__) in name


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The module's file in a folder of its own, older than its sources, and no compiler that works."""
    moe.lib()
    good = build.build_binding()
    path = str(tmp_path / os.path.basename(good))
    with open(good, "rb") as f, open(path, "wb") as to:
        to.write(f.read())
    monkeypatch.setattr(build, "binding_path", lambda: path)
    monkeypatch.setenv("CXX", "/bin/false")
    monkeypatch.setattr(moe, "_native", None)
    return path


def test_stale_module_that_cannot_be_built_is_not_loaded(elsewhere):
    os.utime(elsewhere, (1, 1))
    with pytest.raises(RuntimeError, match="older than its sources"):
        moe._binding()
    assert moe._native is None
    os.unlink(elsewhere)
    with pytest.raises(RuntimeError, match="missing"):
        moe._binding()


def test_fresh_module_needs_no_compiler(elsewhere):
    os.utime(elsewhere, (1 << 33, 1 << 33))
    assert not build.binding_stale()
    assert moe._binding() is moe._native


def test_module_without_its_sources_is_taken_as_it_is(elsewhere, monkeypatch):
    monkeypatch.setattr(build, "BINDING_SOURCE", elsewhere + ".cpp")
    os.utime(elsewhere, (1 << 33, 1 << 33))
    assert moe._binding() is moe._native
