"""A check of the compiler's output for the 4-bit products: no matrix instruction has an
operand in the registers of its accumulators, and operands take 4 registers (e2m1 codes of
128 along k), not 8."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from orthogonalized_updates_amd import build
from test_fp8_assembly_cpu import MFMA, overlapping


def test_matrix_instructions(tmp_path):
    out = tmp_path / "fp4_matmul.s"
    try:
        cc = build.hipcc()
    except RuntimeError:
        pytest.skip("needs hipcc")
    r = subprocess.run([cc, *build.compile_flags(), "--cuda-device-only", "-S", os.path.join(build.CSRC, "fp4_matmul.hip"),
                        "-o", str(out)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    kernel, seen = None, {}
    for line in out.read_text().splitlines():
        label = re.match(r"(_Z\w+):", line)
        if label:
            kernel = label.group(1)
        if re.search(r"\bv_mfma_", line):
            assert overlapping(line) is False, (kernel, line)
            m = MFMA.search(line)
            assert [int(m.group(i + 1)) - int(m.group(i)) for i in (5, 8)] == [3, 3], (kernel, line)
            assert "cbsz:4" in line and "blgp:4" in line
            seen[kernel] = seen.get(kernel, 0) + 1
    for name, n in (("k_matmul4_direct", 2), ("k_matmul4_small", 2), ("k_matmul4_tile", 2), ("k_matmul4_big", 4)):
        assert sum(name in k for k in seen) == n
