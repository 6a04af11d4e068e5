"""A check of the compiler's output for the 8-bit products: no matrix
instruction has an operand in the registers of its accumulators. The compiler
has once placed converted operands there, for a loop written another way, and
results were wrong."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from orthogonalized_updates_amd import build

REGS = r"([va])\[(\d+):(\d+)\]"
# result, two operands, the accumulators it adds to (or a constant)
MFMA = re.compile(rf"v_mfma_\S+ +{REGS}, *{REGS}, *{REGS}, *(?:{REGS}|[-0-9.]+)")
KERNELS = ["k_matmul_direct", "k_matmul_small", "k_matmul_tile", "k_matmul_big"]


def overlapping(line):
    """Whether an operand of a matrix instruction shares registers with the
    accumulators that it adds to: two values in one place. (The result may
    take an operand's place, which is read before.) None for other lines."""
    m = MFMA.search(line)
    if not m:
        return None
    if m.group(10) is None:
        return False
    a, b, acc = ((m.group(i), int(m.group(i + 1)), int(m.group(i + 2))) for i in (4, 7, 10))
    return any(x[0] == acc[0] and x[1] <= acc[2] and acc[1] <= x[2] for x in (a, b))


@pytest.mark.parametrize("line,want", [
    ("\tv_mfma_f32_16x16x32_bf16 v[34:37], v[36:39], v[40:43], v[34:37]", True),
    ("\tv_mfma_f32_16x16x32_bf16 v[34:37], v[40:43], v[33:36], v[34:37]", True),
    ("\tv_mfma_f32_16x16x32_bf16 v[34:37], v[38:41], v[30:33], v[34:37]", False),
    ("\tv_mfma_f32_16x16x32_bf16 a[34:37], v[34:37], v[30:33], a[34:37]", False),
    ("\tv_mfma_f32_16x16x32_bf16 v[34:37], v[34:37], v[30:33], 0", False),
    ("\tv_mfma_f32_16x16x32_bf16 v[18:21], v[18:21], v[22:25], v[26:29]", False),
    ("\tv_mfma_scale_f32_16x16x128_f8f6f4 v[2:5], v[8:15], v[16:23], v[2:5], v161, v146 op_sel_hi:[0,0,0]", False),
    ("\tv_mfma_scale_f32_16x16x128_f8f6f4 v[2:5], v[8:15], v[16:23], 0, v161, v146 op_sel_hi:[0,0,0]", False),
    ("\tv_add_f32 v1, v2, v3", None),
])
def test_the_check_itself(line, want):
    assert overlapping(line) is want


def test_no_operand_lies_over_the_accumulators(tmp_path):
    out = tmp_path / "fp8_matmul.s"
    try:
        cc = build.hipcc()
    except RuntimeError:
        pytest.skip("needs hipcc")
    r = subprocess.run([cc, *build.compile_flags(), "--cuda-device-only", "-S",
                        os.path.join(build.CSRC, "fp8_matmul.hip"), "-o", str(out)],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    kernel, seen, bad = None, {}, []
    for line in out.read_text().splitlines():
        label = re.match(r"(_Z\w+):", line)
        if label:
            kernel = label.group(1)
        if re.search(r"\bv_mfma_", line):
            over = overlapping(line)
            assert over is not None, f"not read: {line}"
            seen[kernel] = seen.get(kernel, 0) + 1
            if over:
                bad.append((kernel, line.strip()))
    assert not bad
    for name in KERNELS:  # 3 instantiations of each, 6 of the largest tiles
        assert sum(name in k for k in seen) == (6 if name == "k_matmul_big" else 3)
