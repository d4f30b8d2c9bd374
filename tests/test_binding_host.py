"""The row operators' compiled binding is optional: a package without it, with one that does not load
or with one of another torch imports and works, and the library builds where it cannot be built."""
import importlib.util
import os
import shutil
import subprocess
import sys
import types

import pytest
import torch

from chunk_causal_wavefront_b200 import rows as PR

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "chunk_causal_wavefront_b200")


@pytest.fixture
def build(monkeypatch, tmp_path):
    """build.py with its binding's outputs in a temporary folder and nothing to compile for the library."""
    spec = importlib.util.spec_from_file_location("wf_build_under_test", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    monkeypatch.setattr(mod, "_compile", lambda src, verbose, extra: mod.LIB)
    monkeypatch.setattr(mod, "BIND", str(tmp_path / os.path.basename(mod.BIND)))
    monkeypatch.setattr(mod, "BUILD", str(tmp_path))
    return mod


USE = """
import warnings
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    import chunk_causal_wavefront_b200 as wf
from chunk_causal_wavefront_b200 import rows
pool = wf.KVPool(wf.make_config(num_stages=2, chunk_tokens=128, num_heads=2, head_dim=128,
                                anchor_chunks=1, history_chunks=1, page_tokens=128))
print(rows._fast is None, sum("_rows_bind" in str(w.message) for w in seen), pool.live_rows)
"""


@pytest.mark.parametrize("module,warned", [(None, 0), (b"not a library", 1)])
def test_package_without_a_module_that_loads(tmp_path, module, warned):
    pkg = tmp_path / "chunk_causal_wavefront_b200"
    pkg.mkdir()
    for f in os.listdir(PKG):
        if f.endswith(".py") or f == "libwf.so":
            shutil.copy(os.path.join(PKG, f), pkg / f)
    if module is not None:
        (pkg / "_rows_bind.so").write_bytes(module)
    r = subprocess.run([sys.executable, "-c", USE], cwd=tmp_path, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == ["True", str(warned), "128"]


def test_module_of_another_torch_is_left_alone(monkeypatch):
    def bind(*addresses):
        raise AssertionError("bound")
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: object())
    for module in (types.SimpleNamespace(torch_version="1.0", bind=bind), types.SimpleNamespace(bind=bind)):
        monkeypatch.setattr(PR.importlib, "import_module", lambda name: module)
        with pytest.warns(RuntimeWarning, match="_rows_bind"):
            assert PR._load_fast() is None


def test_built_module_is_used_and_names_its_torch():
    assert PR._fast is not None and PR._fast.torch_version == torch.__version__


def test_library_builds_without_a_host_compiler(build, monkeypatch, capsys):
    monkeypatch.setenv("CXX", "/bin/false")
    with open(build.BIND, "w") as f:
        f.write("left by an earlier build")
    assert build.build() == build.LIB
    assert "binding was not built" in capsys.readouterr().err
    assert not os.path.exists(build.BIND)                      # it may not fit the library
    monkeypatch.setenv("CXX", "/nowhere/c++")
    assert build.build() == build.LIB


def test_library_builds_without_torch(build, monkeypatch, capsys):
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build.build() == build.LIB
    assert "torch is not installed" in capsys.readouterr().err


def test_module_is_rebuilt_for_another_torch(build, monkeypatch):
    runs = []

    def compiler(cmd, **kw):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("module")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build.subprocess, "run", compiler)
    build.build_bind()
    build.build_bind()
    assert len(runs) == 1
    monkeypatch.setattr(build, "torch_version", lambda d: "99.0")
    build.build_bind()
    assert len(runs) == 2 and '-DWF_TORCH_VERSION="99.0"' in runs[1]


def test_torch_version_is_the_installed_one(build):
    assert build.torch_version(os.path.dirname(torch.__file__)) == torch.__version__
