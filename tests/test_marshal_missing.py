"""The library without the compiled short way into its paged calls: everything is there, through ctypes."""
import os
import subprocess

import pytest
import torch

from draft_tree_build_gb300 import _build, bastion
from test_paged_refusals import _attend, _tensors


@pytest.fixture
def fresh(monkeypatch):
    """A binding that has not loaded its library yet."""
    bastion.lib()
    monkeypatch.setattr(bastion, "_lib", None)
    monkeypatch.setattr(bastion, "_marshal", None)
    return monkeypatch


def _works():
    with pytest.warns(UserWarning, match="ctypes"):
        L = bastion.lib()
    assert bastion._marshal is None
    assert L.bastion_version().startswith(b"bastion-gb300")
    assert bastion.bastion_paged_append_workspace_bytes(4) > 0
    t = _tensors()
    with pytest.raises(bastion.BastionError, match="CUDA device"):  # the last of the binding's own checks
        _attend(bastion, t)
    t["lens"] = t["lens"].long()
    with pytest.raises(bastion.BastionError, match="seq_len"):
        _attend(bastion, t)


def test_no_compiler_and_no_extension(fresh, tmp_path):
    fresh.setattr(_build, "MARSHAL", str(tmp_path / "bastion_marshal.so"))
    run = subprocess.run

    def no_gcc(cmd, *a, **kw):
        if cmd[0] == "gcc":
            raise FileNotFoundError(2, "No such file or directory", "gcc")
        return run(cmd, *a, **kw)

    fresh.setattr(subprocess, "run", no_gcc)
    assert _build.up_to_date()  # the library itself is
    _works()


def test_no_python_headers(fresh, tmp_path):
    fresh.setattr(_build, "MARSHAL", str(tmp_path / "bastion_marshal.so"))
    fresh.setattr(_build.sysconfig, "get_paths", lambda *a, **kw: {"include": str(tmp_path)})
    _works()


def test_a_directory_that_cannot_be_written(fresh, tmp_path):
    fresh.setattr(_build, "MARSHAL", str(tmp_path / "absent" / "bastion_marshal.so"))
    _works()


def test_an_extension_that_does_not_load(fresh, tmp_path):
    so = tmp_path / "bastion_marshal.so"
    so.write_bytes(b"not a shared library")
    fresh.setattr(_build, "MARSHAL", str(so))
    assert _build.marshal_up_to_date()
    _works()


def test_a_torch_without_cuda(fresh):
    fresh.delattr(torch._C, "_cuda_getDevice")
    _works()


def test_an_extension_older_than_its_source_is_not_loaded(fresh, tmp_path):
    so = tmp_path / "bastion_marshal.so"
    so.write_bytes(open(_build.MARSHAL, "rb").read())
    os.utime(so, (0, 0))
    fresh.setattr(_build, "MARSHAL", str(so))
    assert not _build.marshal_up_to_date()
    L = bastion.lib(build_if_missing=False)
    assert bastion._marshal is None and L is bastion.lib()


def test_another_interpreter_has_a_file_of_its_own():
    """The extension is built against one interpreter's C API: another looks for another file, and builds it."""
    import importlib.machinery
    import sys
    import sysconfig
    name = os.path.basename(_build.MARSHAL)
    tag = sysconfig.get_config_var("EXT_SUFFIX")
    assert name == "bastion_marshal" + tag and tag in importlib.machinery.EXTENSION_SUFFIXES
    assert f"{sys.version_info[0]}{sys.version_info[1]}" in tag  # such as .cpython-312-aarch64-linux-gnu.so


def test_a_built_tree_without_its_sources(fresh, tmp_path):
    """The built files alone are enough where nothing is to be built."""
    fresh.setattr(_build, "CSRC", str(tmp_path / "csrc"))
    fresh.setattr(_build, "INCLUDE", str(tmp_path / "include"))
    bastion.lib(build_if_missing=False)
    assert bastion._marshal is not None
