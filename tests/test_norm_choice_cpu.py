"""Which lanes share a row of the RMS norm, built from its own source and run on the host:
launches fit, and the sizes of the GPU tests reach every form, and every form's loop over
further rows."""
from __future__ import annotations

import itertools
import os
import shutil
import subprocess
from collections import namedtuple

import pytest

import orthogonalized_updates_amd as mh

pytest.importorskip("torch")
import test_rms_norm_gpu as tests  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM_INCLUDE = "/opt/rocm/include"
CSRC = f"{ROOT}/orthogonalized_updates_amd/csrc"
Form = namedtuple("Form", "lanes vecs groups rows")
FORWARD = {(16, 1), (64, 1), (64, 2), (64, 3), (256, 1), (256, 2), (256, 4), (1024, 2), (1024, 4), (0, 0)}
BACKWARD = {(16, 1), (64, 1), (64, 2), (64, 3), (64, 4), (256, 2), (256, 4), (1024, 2), (0, 0)}


@pytest.fixture(scope="module")
def forms(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.isdir(ROCM_INCLUDE):
        pytest.skip("needs g++ and the HIP headers")
    exe = tmp_path_factory.mktemp("choice") / "norm_choice"
    cmd = [cxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-D__align__(n)=__attribute__((aligned(n)))", f"-I{CSRC}",
           f"-I{ROOT}/include", f"-I{ROCM_INCLUDE}", f"{ROOT}/tests/host_check/norm_choice.cpp", "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]

    def run(sizes):
        r = subprocess.run([str(exe)], input="".join(f"{a} {b}\n" for a, b in sizes), capture_output=True, text=True, timeout=600)
        assert r.returncode == 0
        got = [list(map(int, line.split())) for line in r.stdout.splitlines()]
        assert len(got) == len(sizes)
        return [(Form(*g[:4]), Form(*g[4:])) for g in got]
    return run


def test_forms_hold_their_rows(forms):
    sizes = list(itertools.product([1, 256, 257, 1 << 20, (1 << 20) + 1, 1 << 24],
                                   [1, 128, 129, 512, 513, 1024, 1025, 1536, 1537, 2048, 2049, 4096, 4097, 8192, 8193, 16384, 16385, 32768, 32769, 1 << 24]))
    for (rows, cols), (f, b) in zip(sizes, forms(sizes)):
        assert (f.lanes, f.vecs) in FORWARD and (b.lanes, b.vecs) in BACKWARD
        for form, longest in ((f, 32768), (b, 16384)):
            assert form.lanes * form.vecs * 8 >= cols if cols <= longest else form.lanes == 0
            assert 1 <= form.groups <= min(1 << 20, -(-rows // form.rows))
        need = b.groups * cols * 4 + (4 * rows if cols > 16384 else 0)
        assert mh.lib.muonh_rms_norm_backward_workspace_bytes(rows, cols) == need


def test_gpu_tests_reach_every_form(forms):
    assert {f[:2] for f, _ in forms(tests.SIZES + tests.LANES_64)} == FORWARD
    assert {b[:2] for _, b in forms(tests.SIZES)} == BACKWARD
    assert {f[:2] for f, _ in forms(tests.LANES_64)} == {(64, 1)}


def test_gpu_tests_reach_every_loop(forms):
    """A workgroup that goes on to further rows. 16 lanes take the most rows that there may be in one turn."""
    turns = {f[:2]: rows - f.groups * f.rows for (rows, _), (f, _) in zip(tests.TALL, forms(tests.TALL))}
    assert set(turns) == FORWARD - {(16, 1)} and all(0 < v < tests.ENDS for v in turns.values())
    assert forms([(1 << 24, 128)])[0][0].groups * 16 == 1 << 24
    back = [(b[:2], rows > b.groups * b.rows) for (rows, _), (_, b) in zip(tests.TURNS, forms(tests.TURNS))]
    assert {form for form, again in back if again} == BACKWARD and all(again for _, again in back)
