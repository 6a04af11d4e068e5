"""A check of the compiler's output where inline asm reads scalar registers: the
LDS DMA's base address must not have been written by a vector instruction in
the 5 cycles before. The compiler keeps that distance for its own memory
instructions, but does not look into inline asm; a base read too early is partly
an older value, and the DMA goes to another address."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from orthogonalized_updates_amd import build

STATES = 5
DMA = re.compile(r"global_load_lds_\w+ v\d+, s\[(\d+):(\d+)\]")


def scalars_written(line):
    """Numbers of the scalar registers that a vector instruction writes."""
    if not line.startswith("v_"):
        return set()
    ops = line.split(None, 1)[1] if " " in line or "\t" in line else ""
    ops = [o.strip() for o in re.split(r",\s*(?![^\[]*\])", ops)]
    # the first operand, and the carry that an add, subtract, multiply-add or division writes second
    outs = ops[:2] if re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co|v_mad_[iu]64|v_div_scale", line) else ops[:1]
    got = set()
    for o in outs:
        m = re.fullmatch(r"s(\d+)|s\[(\d+):(\d+)\]", o)
        if m:
            got |= {int(m.group(1))} if m.group(1) else set(range(int(m.group(2)), int(m.group(3)) + 1))
    return got


def too_early(lines):
    """The DMAs that read a scalar register within STATES wait states of a vector
    instruction's write, in program order."""
    bad, before = [], []
    for line in lines:
        m = DMA.match(line)
        if m:
            read, states = set(range(int(m.group(1)), int(m.group(2)) + 1)), 0
            for b in reversed(before[-2 * STATES:]):
                if states >= STATES:
                    break
                if scalars_written(b) & read:
                    bad.append((b, line))
                    break
                nop = re.match(r"s_nop (\d+)", b)
                states += int(nop.group(1)) + 1 if nop else 1
        before.append(line)
    return bad


def test_the_check_itself():
    dma = "global_load_lds_dwordx4 v3, s[6:7]"
    assert too_early(["v_readfirstlane_b32 s7, v1", "s_nop 0", dma])
    assert too_early(["v_readfirstlane_b32 s6, v1", "s_mov_b32 m0, s1", "s_nop 2", dma])
    assert not too_early(["v_readfirstlane_b32 s6, v1", "s_nop 4", dma])
    assert not too_early(["v_readfirstlane_b32 s8, v1", dma])
    assert not too_early(["s_add_u32 s6, s6, s1", dma])
    assert too_early(["v_cmp_gt_u32_e64 s[6:7], v1, v2", "s_nop 0", dma])
    assert too_early(["v_add_co_u32 v1, s[6:7], v2, v3", dma])
    assert not too_early(["v_mov_b32_e32 v1, s6", dma])


@pytest.mark.parametrize("source", ["fp8_matmul.hip", "fp4_matmul.hip"])
def test_no_dma_reads_its_base_too_early(source, tmp_path):
    out = tmp_path / "out.s"
    try:
        cc = build.hipcc()
    except RuntimeError:
        pytest.skip("needs hipcc")
    r = subprocess.run([cc, *build.compile_flags(), "--cuda-device-only", "-S", os.path.join(build.CSRC, source), "-o", str(out)],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    lines = [t for t in (l.strip() for l in out.read_text().splitlines()) if t and not t.startswith((".", ";")) and not t.endswith(":")]
    assert sum(bool(DMA.match(l)) for l in lines) > 100  # the regular expression still finds them
    assert sum("global_load_lds" in l for l in lines) == sum(bool(DMA.match(l)) for l in lines)
    assert not too_early(lines)
