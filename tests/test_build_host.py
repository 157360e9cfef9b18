"""The build of the package's two binaries: the library with the C ABI, and the
C++ module with the training operators' allocating wrappers, which needs a host
compiler, Python's and torch's headers."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

from flash_mixed_chunk_gb300 import _buildlib

CODE = """
import torch
import flash_mixed_chunk_gb300 as fm
assert fm.flash_mca_version() and fm.flash_mca_workspace_bytes(1, 512, 128, 256, 256, True, 1) > 0
assert fm.flash_mca_layer_norm_backward_workspace_bytes(4, 8) > 0
x, w = torch.zeros(2, 8), torch.zeros(8)
for call in (lambda: fm.layer_norm(x, w, w), lambda: fm.vocab_loss(x, x, w)):
    try:
        call()
    except ImportError as e:
        assert "binding" in str(e) and "g++" in str(e), e
    else:
        raise SystemExit("no error")
print("fine")
"""


def test_the_core_needs_the_library_alone(tmp_path):
    """Without a host compiler and without the module the package imports, its
    other calls work, and the wrappers say what is missing."""
    root = os.path.dirname(_buildlib.PKG)
    for part in ("flash_mixed_chunk_gb300", "include"):
        shutil.copytree(os.path.join(root, part), tmp_path / part,
                        ignore=shutil.ignore_patterns("_binding*", "_build", "__pycache__"))
    (tmp_path / "bin").mkdir()
    env = {**os.environ, "PATH": str(tmp_path / "bin")}
    env.pop("PYTHONPATH", None)
    p = subprocess.run([sys.executable, "-c", CODE], cwd=tmp_path, env=env, capture_output=True,
                       text=True, timeout=300)
    assert p.returncode == 0 and "fine" in p.stdout, p.stderr[-2000:]


def test_the_module_belongs_to_one_python_and_torch(monkeypatch):
    """Its file carries Python's ABI tag, and another torch makes it out of date
    whatever the files' times are."""
    import sysconfig

    import torch
    assert os.path.basename(_buildlib.BINDING) == "_binding" + sysconfig.get_config_var("EXT_SUFFIX")
    _buildlib.build()
    assert not _buildlib._binding_stale()
    monkeypatch.setattr(torch, "__version__", "1.0")
    assert _buildlib._binding_stale()
    monkeypatch.undo()
    monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    assert _buildlib._binding_stale()
    monkeypatch.undo()
    assert not _buildlib._binding_stale()


def copied(tmp_path, ignore):
    root = os.path.dirname(_buildlib.PKG)
    for part in ("flash_mixed_chunk_gb300", "include"):
        shutil.copytree(os.path.join(root, part), tmp_path / part,
                        ignore=shutil.ignore_patterns("__pycache__", *ignore))
    (tmp_path / "bin").mkdir()
    env = {**os.environ, "PATH": str(tmp_path / "bin")}
    env.pop("PYTHONPATH", None)

    def python(code):
        return subprocess.run([sys.executable, "-c", code], cwd=tmp_path, env=env,
                              capture_output=True, text=True, timeout=300)
    return python


def test_a_tree_without_its_build_folder_is_not_built_again(tmp_path):
    """Both binaries and what they were built against are all that a copy of the
    package needs: no compiler, no folder of objects."""
    _buildlib.build()
    p = copied(tmp_path, ["_build"])("""
import torch
import flash_mixed_chunk_gb300 as fm
try:
    fm.layer_norm(torch.zeros(2, 8), torch.zeros(8), torch.zeros(8))
except ValueError as e:
    assert "CUDA" in str(e)
    print("fine")
""")
    assert p.returncode == 0 and "fine" in p.stdout, p.stderr[-2000:]
    assert not (tmp_path / "flash_mixed_chunk_gb300" / "_build").exists()


def test_a_module_that_cannot_be_built_for_want_of_a_folder(tmp_path):
    python = copied(tmp_path, ["_build", "_binding*"])
    (tmp_path / "flash_mixed_chunk_gb300" / "_build").write_text("not a folder")
    p = python(CODE)
    assert p.returncode == 0 and "fine" in p.stdout, p.stderr[-2000:]
