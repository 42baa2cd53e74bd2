"""The extension module of the batch operators' binding: what needs it, and what does not (CPU only)."""

import os
import subprocess
import sys
import sysconfig

import pytest

pytest.importorskip("int4_blockwise_quantised_b200._vv")
from int4_blockwise_quantised_b200 import build  # noqa: E402


def copy_without_marshal(tmp_path):
    """The package in a folder of its own, with libvv.so and without _marshal."""
    pkg = tmp_path / os.path.basename(build.PKG)
    pkg.mkdir()
    for f in os.listdir(build.PKG):
        if f.endswith(".py"):
            (pkg / f).write_bytes(open(os.path.join(build.PKG, f), "rb").read())
    os.symlink(build.LIB, pkg / "libvv.so")
    os.symlink(build.INCLUDE, tmp_path / "include")
    return pkg


def test_other_operators_need_no_marshal(tmp_path):
    pkg = copy_without_marshal(tmp_path)
    code = f"""
from {pkg.name} import _vv
assert _vv.__file__.startswith({str(tmp_path)!r})
assert _vv.vv_version() and _vv.vv_gqa_prefix_attn_workspace_size(2, 4, 2, 128, 100, 64) > 0
for call in (lambda: _vv.vv_paged_plan(*[None] * 7), lambda: _vv.vv_logits_process(None)):
    try:
        call()
    except ImportError as e:
        assert "_marshal" in str(e) and "build" in str(e)
    else:
        raise AssertionError("no ImportError")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_build_makes_the_library_without_marshal(monkeypatch):
    def fail(*a):
        raise RuntimeError("no host compiler")

    monkeypatch.setattr(build, "_compile_marshal", fail)
    assert build.build(lib_only=True) == build.LIB
    with pytest.raises(RuntimeError, match="libvv.so is built"):
        build.build()


def test_module_is_of_this_python():
    assert build.MARSHAL.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and os.path.exists(build.MARSHAL)
    assert not os.path.exists(os.path.join(build.PKG, "_marshal.so"))  # another Python would load it


def test_module_is_built_again_for_another_torch(monkeypatch):
    ran = []

    def run(cmd, **k):
        ran.append(cmd)
        return subprocess.CompletedProcess(cmd, 1, "", "not run")

    build._compile_marshal(False)
    monkeypatch.setattr(build.subprocess, "run", run)
    build._compile_marshal(False)
    assert not ran  # up to date
    monkeypatch.setattr(build, "_made_for", lambda: "another torch")
    with pytest.raises(RuntimeError):
        build._compile_marshal(False)
    assert len(ran) == 1 and ran[0][0] == "g++"


def test_module_made_for_another_torch_is_not_used(tmp_path):
    pkg = copy_without_marshal(tmp_path)
    os.symlink(build.MARSHAL, pkg / os.path.basename(build.MARSHAL))
    code = f"""
import torch
torch.__version__ = "1.2.3+cu0"
from {pkg.name} import _vv
try:
    _vv.vv_logits_process(None)
except ImportError as e:
    assert "1.2.3" in str(e)
else:
    raise AssertionError("no ImportError")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
