"""Host-only checks of the binding's C++ part: the package works without it, takes
none that was built for another torch, and builds it anew when torch or Python change."""
import importlib.machinery
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "bidirectional_mamba_ssd_b200"
USE = """
import warnings
with warnings.catch_warnings(record=True) as w:
    warnings.simplefilter("always")
    import bidirectional_mamba_ssd_b200 as ssd
from bidirectional_mamba_ssd_b200 import causal
assert ssd.lib.ssd_version() >= 100 and ssd.ssd_workspace_bytes(0, 2, 300, 4, 64, 128, 2, 64, 1) > 256
assert any("binding is not used" in str(m.message) for m in w), [str(m.message) for m in w]
assert causal._binding.causal_step() is NotImplemented
import torch
for call in (lambda: ssd.ssd_causal_step(*[torch.zeros(1, 1, 64)] * 7), lambda: ssd.ssd_cache_copy(None, None, None)):
    try:
        call()
    except (TypeError, ValueError):
        continue
    raise AssertionError("a call of CPU tensors is refused")
"""


@pytest.mark.parametrize("there", ["nothing", "not_a_module", "another_torch", "without_a_version"])
def test_package_without_the_extension(tmp_path, there):
    import __graft_entry__
    __graft_entry__.build()
    pkg = tmp_path / PKG
    pkg.mkdir()
    for name in os.listdir(os.path.join(ROOT, PKG)):
        if name.endswith(".py"):
            shutil.copy(os.path.join(ROOT, PKG, name), pkg / name)
    os.symlink(os.path.join(ROOT, PKG, "libssd_bidir.so"), pkg / "libssd_bidir.so")
    if there == "not_a_module":
        (pkg / "_binding.so").write_bytes(b"no ELF file")
    elif there == "another_torch":
        (pkg / "_binding.py").write_text("torch_version = '1.0'\ndef setup(*a):\n    raise RuntimeError('used')\n")
    elif there == "without_a_version":
        (pkg / "_binding.py").write_text("def setup(*a):\n    raise RuntimeError('used')\n")
    done = subprocess.run([sys.executable, "-c", USE], cwd=tmp_path, capture_output=True, text=True, timeout=300,
                          env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert done.returncode == 0, done.stderr[-2000:]


def test_extension_is_built_anew_for_another_torch(tmp_path, monkeypatch):
    spec = importlib.util.spec_from_file_location("build_under_test", os.path.join(ROOT, PKG, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    assert importlib.machinery.EXTENSION_SUFFIXES[0] == os.path.basename(b.BINDING)[len("_binding"):]
    monkeypatch.setattr(b, "PKG", str(tmp_path))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so_tagged"))
    monkeypatch.setattr(b, "BINDING_KEY", str(tmp_path / "_binding.key"))
    runs = []

    def run(cmd, check):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass

    monkeypatch.setattr(b.subprocess, "run", run)
    (tmp_path / "_binding.so").write_text("of an earlier build")
    b.build_binding()
    assert len(runs) == 1 and not (tmp_path / "_binding.so").exists()
    b.build_binding()
    assert len(runs) == 1
    monkeypatch.setattr(b, "_torch_version", lambda: "99.0")
    b.build_binding()
    assert len(runs) == 2 and '-DSSD_TORCH_VERSION="99.0"' in runs[1]
    b.build_binding()
    assert len(runs) == 2
    monkeypatch.setattr(b.sys, "version", "another Python")
    b.build_binding()
    assert len(runs) == 3
    (tmp_path / "_binding.key").unlink()
    b.build_binding()
    assert len(runs) == 4
