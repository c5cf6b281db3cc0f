"""The package with one of its two compiled files missing, broken or built against another torch: without the
library it does not import, without the binding only the binding's own entry points fail, and the message names the
file (CPU only)."""
import os
import shutil
import subprocess
import sys

import pytest

import block_scaled_fp8_gemm_gb300 as g

PKG = os.path.dirname(os.path.abspath(g.__file__))
NAME = os.path.basename(PKG)


@pytest.fixture
def copy(tmp_path):
    """The package's files in a folder of their own, the library as a link."""
    to = tmp_path / NAME
    to.mkdir()
    for f in ("__init__.py", "build.py"):
        shutil.copy(os.path.join(PKG, f), to / f)
    for f in ("libgemmar.so", "_operators.so"):
        os.symlink(os.path.join(PKG, f), to / f)
    return to


def run(copy, code):
    r = subprocess.run([sys.executable, "-c", code], cwd=copy.parent, capture_output=True, text=True,
                       env={k: v for k, v in os.environ.items() if k != "PYTHONPATH"})
    return r.returncode, r.stdout + r.stderr


USE = f"""
import inspect
import types
import {NAME} as g
ctx = types.SimpleNamespace(handle=types.SimpleNamespace(value=None))
assert g.gemmar_supports(1, 128, 256, 128, 1, 0) == 0   # the library itself is there
for name in ("norm_gate_residual", "norm_gate_residual_bwd", "lora_apply", "lora_apply_bwd"):
    f = getattr(g, name)
    try:
        f(ctx, *[None] * (sum(p.default is p.empty for p in inspect.signature(f).parameters.values()) - 1), stream=0)
    except ImportError as e:
        print(e)
"""


def test_both_files(copy):
    rc, out = run(copy, f"import {NAME} as g; print(g._operators.torch_version)")
    assert rc == 0 and out.strip() == __import__("torch").__version__


def test_no_library(copy):
    (copy / "libgemmar.so").unlink()
    rc, out = run(copy, f"import {NAME}")
    assert rc != 0 and "libgemmar.so not found" in out


def test_no_binding(copy):
    (copy / "_operators.so").unlink()
    rc, out = run(copy, USE)
    assert rc == 0 and out.count("_operators.so not found") == 4, out


def test_a_binding_that_does_not_load(copy):
    (copy / "_operators.so").unlink()
    (copy / "_operators.so").write_bytes(b"no shared object")
    rc, out = run(copy, USE)
    assert rc == 0 and out.count("does not load") == 4 and "_operators.so" in out, out


def test_a_binding_of_another_torch(copy):
    rc, out = run(copy, "import torch\ntorch.__version__ = '0.0.1'\n" + USE)
    assert rc == 0 and out.count("was built against torch") == 4 and "0.0.1" in out, out
