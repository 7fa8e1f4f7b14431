"""The package imports, checks its tensors and builds without the native checks of csrc/args.c (no GPU needed)."""
import importlib.util
import os
import subprocess
import sys

import pytest

pytest.importorskip("kpool_indexer_int8_b200")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
IMPORT = """
import torch
import kpool_indexer_int8_b200 as kp
assert kp._args is None
z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt)
try:
    kp._take(0, (z(2),), (torch.int32,), ((2,),), ("length",))
except ValueError as e:
    assert "length must be a CUDA tensor" in str(e)
else:
    raise AssertionError("a CPU tensor was taken")
print("checked")
"""


@pytest.mark.parametrize("before", [
    "import sys; sys.modules['kpool_indexer_int8_b200._args'] = None",      # not built, or for another Python
    # a torch without the exchange table, or of another version of it
    "import sys, types; m = sys.modules['kpool_indexer_int8_b200._args'] = types.ModuleType('_args')\n"
    "def setup(*a): raise AttributeError('__dlpack_c_exchange_api__')\nm.setup = setup",
    "import sys, types; m = sys.modules['kpool_indexer_int8_b200._args'] = types.ModuleType('_args')\n"
    "def setup(*a): raise ImportError('DLPack 2')\nm.setup = setup",
], ids=["missing", "no table", "another version"])
def test_import_without_the_native_checks(before):
    r = subprocess.run([sys.executable, "-c", before + IMPORT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "checked" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("missing", ["compiler", "torch"])
def test_the_library_builds_without_them(missing, monkeypatch, tmp_path, capsys):
    spec = importlib.util.spec_from_file_location("_build_alone", os.path.join(ROOT, "kpool_indexer_int8_b200", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    monkeypatch.setattr(mod, "ARGS_LIB", str(tmp_path / "_args.so"))
    if missing == "compiler":
        monkeypatch.setenv("CC", str(tmp_path / "no-such-compiler"))
    else:
        find = importlib.util.find_spec
        monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    # (the library's own objects are taken as built: nothing is compiled or linked here)
    monkeypatch.setattr(mod, "_headers_mtime", lambda: 0.0)
    monkeypatch.setattr(mod.glob, "glob", lambda pattern: [])
    monkeypatch.setattr(mod, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(mod.subprocess, "run", run_linker(mod.subprocess.run, tmp_path))
    assert mod.build() == str(tmp_path / "lib.so") and os.path.exists(tmp_path / "lib.so")
    assert "_args.so is not built" in capsys.readouterr().err and not os.path.exists(tmp_path / "_args.so")


def run_linker(run, tmp_path):
    def fake(cmd, **kw):
        if "-shared" in cmd and "-cudart" in cmd:
            (tmp_path / "lib.so.tmp").write_text("")
            return subprocess.CompletedProcess(cmd, 0, "", "")
        return run(cmd, **kw)
    return fake
