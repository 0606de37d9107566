"""The convolution does not need the dense library: the package imports and
plans without it, and the dense entries say what is missing when asked for."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code, **env):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=dict(os.environ, **env), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return r.stdout


PLAN = """
import sys
import torch
import int8_convolution_forward_amd as ci8
from int8_convolution_forward_amd import *
x, w = torch.zeros(1, 16, 8, 8, dtype=torch.int8), torch.zeros(16, 16, 3, 3, dtype=torch.int8)
assert "tile=" in conv_fprop_i8_plan(x, w, padding=1)
"""


def test_convolution_without_the_dense_library():
    out = run(PLAN + """
assert "int8_convolution_forward_amd.dense" not in sys.modules
for ask in (lambda: ci8.linear, lambda: ci8.dense, lambda: __import__("int8_convolution_forward_amd.dense")):
    try:
        ask()
    except ImportError as e:
        print(e)
""", CONV_I8_DENSE_LIB="/nonexistent/libdense.so")
    assert out.count("/nonexistent/libdense.so is not built") == 3


def test_dense_names_are_there_at_their_first_use():
    run("""
import sys
import int8_convolution_forward_amd as ci8
assert "int8_convolution_forward_amd.dense" not in sys.modules
assert "linear" in dir(ci8) and "layer_norm" in ci8.__all__
assert ci8.linear is ci8.dense.linear and ci8.layer_norm_i8 is ci8.dense.layer_norm_i8
from int8_convolution_forward_amd import *
assert linear is ci8.linear
try:
    ci8.no_such_name
except AttributeError as e:
    assert "no_such_name" in str(e)
else:
    raise AssertionError
""")


def test_a_failed_dense_build_leaves_the_convolution(tmp_path, monkeypatch):
    """Commands that only copy and fail stand for the compilers."""
    import pytest

    from int8_convolution_forward_amd import build

    for name in ("LIB", "DENSE_LIB", "DENSE_BIND"):
        monkeypatch.setattr(build, name, str(tmp_path / name))
    monkeypatch.setattr(build, "LIB_DIR", str(tmp_path))
    compiler = tmp_path / "hipcc"
    compiler.write_text("#!/bin/sh\nfor a; do [ \"$last\" = -o ] && echo built > \"$a\"; last=$a; done\n")
    compiler.chmod(0o755)
    monkeypatch.setattr(build, "HIPCC", str(compiler))
    monkeypatch.setattr(build, "bind_command", lambda out: ["false"])
    with pytest.raises(RuntimeError, match="the compiler failed"):
        build.build()
    assert (tmp_path / "LIB").read_text() == "built\n"
    assert not (tmp_path / "DENSE_LIB").exists() and not (tmp_path / "DENSE_BIND").exists()
