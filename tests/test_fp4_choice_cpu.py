"""The rule that chooses a kernel for a 4-bit product, built from its own source and
run on the host: its launches fit, and the sizes of the GPU tests reach every
kernel that it chooses between."""
from __future__ import annotations

import itertools
import os
import random
import shutil
import subprocess
from collections import namedtuple

import pytest

pytest.importorskip("torch")
import test_fp4_gpu  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM_INCLUDE = "/opt/rocm/include"
CSRC = f"{ROOT}/orthogonalized_updates_amd/csrc"
MAX_DIM, MAX_TILES = 1 << 24, (1 << 21) - 8
Choice = namedtuple("Choice", "em en splits per ws blocks")


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.isdir(ROCM_INCLUDE):
        pytest.skip("needs g++ and the HIP headers")
    exe = tmp_path_factory.mktemp("choice") / "fp4_choice"
    cmd = [cxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-D__align__(n)=__attribute__((aligned(n)))", f"-I{CSRC}",
           f"-I{ROOT}/include", f"-I{ROCM_INCLUDE}", f"{ROOT}/tests/host_check/fp4_choice.cpp", "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]

    def run(sizes):
        text = "\n".join(" ".join(map(str, s)) for s in sizes) + "\n"
        r = subprocess.run([str(exe)], input=text, capture_output=True, text=True, timeout=600)
        assert r.returncode == 0
        got = [Choice(*map(int, line.split())) for line in r.stdout.splitlines()]
        assert len(got) == len(sizes)
        return got
    return run


def up(v, m):
    return -(-v // m)


def test_launches_fit(choose):
    edge = [1, 15, 16, 17, 64, 65, 128, 129, 256, 1 << 14, (1 << 14) + 1, 1 << 20, MAX_DIM - 1, MAX_DIM]
    rng = random.Random(7)
    sizes = list(itertools.product(edge, edge, [0, 1, 256, 257, 1000, 1 << 16, 1 << 23, MAX_DIM]))
    sizes += [tuple(min(MAX_DIM, int(2 ** rng.uniform(0, 24.001))) for _ in range(3)) for _ in range(4000)]
    sizes = [s for s in sizes if up(s[0], 128) * up(s[1], 128) <= MAX_TILES]
    for (m, n, k), c in zip(sizes, choose(sizes)):
        assert c.blocks * 512 < 1 << 32, (m, n, k, c)
        nkb = up(k, 256)
        if c.splits > 1:
            assert (c.splits - 1) * c.per < nkb <= c.splits * c.per and c.em == 64
            assert c.ws == 4 * c.splits * m * up(n, 4) * 4
        else:
            assert c.ws == 0 and c.per == nkb
        # 32-bit offsets within a tile's rows: 256 of less than 2^23 bytes, 64 of at most 2^23
        assert c.em <= 64 or nkb * 128 < 1 << 23


def kernel(c):
    return {(16, 16): "16", (64, 64): "64 split" if c.splits > 1 else "64", (128, 128): "128", (192, 256): "192 x 256",
            (256, 256): "256"}[c.em, c.en]


def sizes_of(test):
    return next([tuple(p[:3]) for p in mark.args[1]] for mark in test.pytestmark
                if mark.name == "parametrize" and mark.args[0].startswith("m,n,k"))


@pytest.mark.parametrize("test", ["test_product_exact", "test_product", "test_small_sums_survive_large_products_that_cancel",
                                  "test_nan_groups_stay_in_their_rows", "test_output_rows_inside_wider_ones"])
def test_gpu_tests_reach_every_kernel(choose, test):
    got = {kernel(c) for c in choose(sizes_of(getattr(test_fp4_gpu, test)))}
    assert got == {"16", "64", "64 split", "128", "192 x 256", "256"}


def test_loop_lengths(choose):
    """1 to 5 blocks of k, and more, at each of the large tiles: their loops' first and last turns are code of their own."""
    seen = {}
    for m, n, k in sizes_of(test_fp4_gpu.test_product_exact):
        seen.setdefault(kernel(choose([(m, n, k)])[0]), set()).add(min(up(k, 256), 6))
    for name in ("128", "192 x 256", "256"):
        assert seen[name] >= {1, 2, 3, 4, 5, 6}, (name, seen[name])
