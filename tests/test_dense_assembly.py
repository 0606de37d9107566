"""The product kernel's matrix instructions are written as such, so the compiler
neither keeps their operands' hazards nor waits for their results: checked here
on the assembly it makes of the kernel."""
import os
import re
import subprocess

import pytest

from int8_convolution_forward_amd import build

SOURCES = [s for s in build.DENSE_SOURCES if os.path.basename(s).startswith("gemm_")]
# A vector instruction's result needs two wait states before a matrix instruction
# reads it; a 16x16 product is in its registers after at most 18.
BEFORE, AFTER = 2, 18


def registers(operand):
    m = re.match(r"-?\|?([va])\[(\d+):(\d+)\]", operand)
    if m:
        return {(m[1], i) for i in range(int(m[2]), int(m[3]) + 1)}
    m = re.match(r"-?\|?([va])(\d+)\b", operand)
    return {(m[1], int(m[2]))} if m else set()


def hazards(lines):
    """(matrix instructions, what comes too soon before or after one), in the order of the text."""
    found, products, at = [], 0, 0
    made, written = {}, {}  # register -> position of the product, of the vector instruction, that writes it
    for line in lines:
        line = line.split(";")[0].strip()
        if line.startswith("_Z") and line.endswith(":"):
            made, written = {}, {}
        op, _, rest = line.partition(" ")
        op, _, tab = op.partition("\t")
        if not re.match(r"(v|s|ds|buffer|global|flat)_", op):
            continue
        operands = [t.strip() for t in (tab + rest).split(",")]
        at += 1 + (int(operands[0]) if op == "s_nop" else 0)
        if op.startswith("v_mfma"):
            products += 1
            for r in set().union(*map(registers, operands[1:4])):
                if at - written.get(r, -99) <= BEFORE:
                    found.append(line)
            for r in registers(operands[0]):
                made[r] = at
        else:
            used = set().union(*map(registers, operands))
            if any(at - made.get(r, -99) <= AFTER for r in used):
                found.append(line)
            if op.startswith("v_"):
                for r in registers(operands[0]):
                    made.pop(r, None)
                    written[r] = at
    return products, found


def test_the_check_sees_a_hazard():
    text = ["v_mov_b32_e32 v4, 0", "v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[8:11], a[0:3]",
            "s_nop 15", "v_accvgpr_read_b32 v1, a2"]
    assert hazards(text) == (1, [text[1], text[3]])
    clean = [text[0], "s_nop 1", text[1], "s_nop 15", "s_nop 15", text[3]]
    assert hazards(clean) == (1, [])


@pytest.mark.slow
def test_products_have_their_wait_states(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    flags = [f for f in build.HIP_FLAGS if f != "-shared"]
    running = []
    for s in SOURCES:
        out = str(tmp_path / (os.path.basename(s) + ".s"))
        running.append((out, subprocess.Popen([build.HIPCC, *flags, "--offload-device-only", "-S", "-I", build.INCLUDE, "-I",
                                               build.DENSE_CSRC, s, "-o", out], stderr=subprocess.PIPE, text=True)))
    for out, p in running:
        _, err = p.communicate()
        assert p.returncode == 0, err[-4000:]
        products, found = hazards(open(out))
        assert products >= 200 and not found, (out, found[:5])
