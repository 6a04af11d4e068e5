"""How the embedding gradient is taken apart, built from its own source and run on the
host: its launches fit, and the sizes of the GPU tests reach every kernel, length of a
chunk and form of the joining."""
from __future__ import annotations

import itertools
import os
import shutil
import subprocess
from collections import namedtuple

import pytest

import orthogonalized_updates_amd as mh

pytest.importorskip("torch")
import test_embedding_gpu  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM_INCLUDE = "/opt/rocm/include"
CSRC = f"{ROOT}/orthogonalized_updates_amd/csrc"
Plan = namedtuple("Plan", "lanes slabs chunk chunks waves bytes")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.isdir(ROCM_INCLUDE):
        pytest.skip("needs g++ and the HIP headers")
    exe = tmp_path_factory.mktemp("plan") / "embedding_plan"
    cmd = [cxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-D__align__(n)=__attribute__((aligned(n)))", f"-I{CSRC}",
           f"-I{ROOT}/include", f"-I{ROCM_INCLUDE}", f"{ROOT}/tests/host_check/embedding_plan.cpp", "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]

    def run(sizes):
        r = subprocess.run([str(exe)], input="".join(f"{n} {cols}\n" for n, cols in sizes), capture_output=True, text=True, timeout=600)
        assert r.returncode == 0
        got = [Plan(*map(int, line.split())) for line in r.stdout.splitlines()]
        assert len(got) == len(sizes)
        return got
    return run


def up(v, m):
    return -(-v // m)


def test_launches_fit(plan):
    sizes = [(n, c) for n, c in itertools.product([1, 1000, 1024, 1025, 4096, 16385, 32768, 32769, 1 << 20, 1 << 24],
                                                  [1, 128, 129, 512, 513, 2048, 40000, 1 << 20, 1 << 24]) if n * c <= 1 << 38]
    for (n, cols), p in zip(sizes, plan(sizes)):
        assert p.bytes == mh.lib.muonh_embedding_backward_workspace_bytes(n, cols)
        if p.lanes == 0:
            assert n <= 1024 and (n * up(cols, 512) + 2048) * 256 < 1 << 32
            continue
        assert p.lanes * 8 * p.slabs >= cols and (p.chunks - 1) * p.chunk < n <= p.chunks * p.chunk
        assert up(p.chunks * p.slabs, 256 // p.lanes) * 256 < 1 << 32  # k_sums
        assert (p.chunks - 2) * p.slabs * 64 * p.waves < 1 << 32       # k_join
        assert p.waves == (8 if p.slabs == 1 else 4) and (p.lanes == 64 or p.waves == 8)


def test_gpu_tests_reach_every_kernel(plan):
    sizes = [(n, cols) for n, _, cols in test_embedding_gpu.SIZES + test_embedding_gpu.MORE_SIZES]
    assert any(p.lanes == 0 for p in plan(sizes))
    joined = {(p.lanes, p.waves) for p in plan(sizes) if p.chunks > 2}
    assert joined == {(16, 8), (64, 8), (64, 4)}
    assert {p.chunk for p in plan(sizes) if p.lanes == 16} >= {4, 8, 16}
    assert {p.chunk for p in plan(sizes) if p.lanes == 64 and p.slabs == 1} >= {4, 8, 16}
    assert {p.chunk for p in plan(sizes) if p.lanes == 64 and p.slabs > 1} >= {4, 8, 16, 32}
    # last chunks that are whole and last chunks that are not, at each number of lanes
    for lanes in (16, 64):
        assert {n % p.chunk == 0 for (n, _), p in zip(sizes, plan(sizes)) if p.lanes == lanes} == {True, False}
