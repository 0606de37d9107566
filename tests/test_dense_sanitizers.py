"""The dense entries' host side (argument checks, plans, workspace sizes) under
AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU: a build of the host
pass only, whose device code is an empty stand-in, against
tests/test_dense_boundary.py loaded through CONV_I8_DENSE_LIB."""
import os
import subprocess
import sys

import pytest

from int8_convolution_forward_amd import build
from tests.test_host_sanitizers import CLANG, HERE, HIPCC, SAN_ENV, _run_clean, _runtime


def test_dense_host_side_under_asan_ubsan(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("no hipcc")
    rt = _runtime(CLANG, "libclang_rt.asan-x86_64.so")
    if rt is None:
        pytest.skip("clang has no AddressSanitizer runtime here")
    objects, running = [], []
    for source in build.DENSE_SOURCES:
        objects.append(str(tmp_path / (os.path.basename(source) + ".o")))
        running.append(subprocess.Popen(
            [HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g", "-std=c++17", "-fPIC", "-w",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=undefined",
             "-I", build.INCLUDE, "-I", build.DENSE_CSRC, "-c", source, "-o", objects[-1]],
            stderr=subprocess.PIPE, text=True))
    for p in running:
        _, err = p.communicate()
        assert p.returncode == 0, err[-4000:]
    # the objects name their device code, which a host-only build does not have
    names = subprocess.run(["nm", "-u", *objects], capture_output=True, text=True, check=True).stdout.split()
    stub = tmp_path / "stub.c"
    stub.write_text("".join(f"const char {n}[4096] __attribute__((aligned(4096))) = {{0}};\n"
                            for n in sorted(set(names)) if n.startswith("__hip_fatbin_")))
    lib = str(tmp_path / "libdense_asan.so")
    r = subprocess.run([CLANG, "-shared", "-fPIC", "-fsanitize=address,undefined", "-shared-libsan", str(stub), *objects,
                        "-o", lib, "-L", "/opt/rocm/lib", "-lamdhip64", "-lstdc++"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, LD_PRELOAD=rt, CONV_I8_DENSE_LIB=lib, **SAN_ENV)
    env.pop("CONV_I8_DENSE_TILE", None)
    out = _run_clean([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                      os.path.join(HERE, "test_dense_boundary.py")], env)
    assert " passed" in out and " failed" not in out
