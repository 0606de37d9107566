"""The scaled matrix instructions of the product kernel for 8-bit floating point,
written as such, have their wait states: their scales as well as the registers that
test_dense_assembly checks."""
import os
import re
import subprocess

import pytest

from int8_convolution_forward_amd import build
from tests.test_dense_assembly import AFTER, BEFORE, hazards, registers


def scale_hazards(lines):
    """(scaled instructions, those whose scales a vector instruction wrote too shortly before)."""
    found, products, at, written = [], 0, 0, {}
    for line in lines:
        line = line.split(";")[0].strip()
        if line.startswith("_Z") and line.endswith(":"):
            written = {}
        m = re.match(r"((?:v|s|ds|buffer|global|flat|scratch)_\w+)\s*(.*)", line)
        if not m:
            continue
        op, operands = m[1], [t.strip() for t in m[2].split(",")]
        at += 1 + (int(operands[0]) if op == "s_nop" else 0)
        if op.startswith("v_mfma_scale"):
            products += 1
            scales = [operands[4], operands[5].split()[0]]
            if any(at - written.get(r, -99) <= BEFORE for s in scales for r in registers(s)):
                found.append(line)
        elif op.startswith("v_") and not op.startswith("v_mfma"):
            for r in registers(operands[0]):
                written[r] = at
    return products, found


def test_the_check_sees_a_hazard():
    mfma = "v_mfma_scale_f32_16x16x128_f8f6f4 a[0:3], v[4:11], v[12:19], a[0:3], v20, v21 op_sel_hi:[0,0,0]"
    text = ["v_alignbyte_b32 v20, v20, v20, 1", mfma]
    assert scale_hazards(text) == (1, [mfma])
    assert scale_hazards([text[0], "s_nop 1", mfma]) == (1, [])
    assert scale_hazards(["v_mov_b32_e32 v21, 0", "s_nop 0", mfma]) == (1, [mfma])
    assert AFTER >= 11 + 2  # eight passes of the matrix unit


@pytest.mark.slow
def test_scaled_products_have_their_wait_states(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    source = next(s for s in build.DENSE_SOURCES if os.path.basename(s) == "gemm_f8.hip")
    flags = [f for f in build.HIP_FLAGS if f != "-shared"]
    out = str(tmp_path / "gemm_f8.s")
    r = subprocess.run([build.HIPCC, *flags, "--offload-device-only", "-S", "-I", build.INCLUDE, "-I", build.DENSE_CSRC, source,
                        "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    lines = open(out).read().split("\n")
    for products, found in (scale_hazards(lines), hazards(lines)):
        assert products >= 200 and not found, found[:5]
