"""The rule that chooses a kernel for a block-scaled product, built from its
own source and run on the host: its launches fit whatever its constants say,
and the sizes of the GPU tests reach every kernel that it chooses between."""
from __future__ import annotations

import itertools
import os
import random
import shutil
import subprocess
from collections import namedtuple

import pytest

pytest.importorskip("torch")
import test_fp8_ends_gpu  # noqa: E402
import test_fp8_gpu  # noqa: E402
import test_fp8_split_gpu  # noqa: E402
import test_fp8_sums_gpu  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM_INCLUDE = "/opt/rocm/include"
CSRC = f"{ROOT}/orthogonalized_updates_amd/csrc"
MAX_DIM, MAX_TILES = 1 << 24, (1 << 21) - 8
Choice = namedtuple("Choice", "em en splits per ws blocks")


def build(where, header=None):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.isdir(ROCM_INCLUDE):
        pytest.skip("needs g++ and the HIP headers")
    if header is not None:
        (where / "fp8_choice.h").write_text(header)
    exe = where / "fp8_choice"
    cmd = [cxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-D__align__(n)=__attribute__((aligned(n)))",
           f"-I{where}", f"-I{CSRC}", f"-I{ROOT}/include", f"-I{CSRC}/../../include", f"-I{ROCM_INCLUDE}",
           f"{ROOT}/tests/host_check/fp8_choice.cpp", "-o", str(exe)]
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


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    return build(tmp_path_factory.mktemp("choice"))


def up(v, m):
    return -(-v // m)


def far_sizes():
    """Accepted products of extreme and random sizes, in both orientations."""
    edge = [1, 15, 16, 17, 32, 33, 48, 64, 65, 128, 129, 256, 1 << 14, (1 << 14) + 1, 1 << 20, MAX_DIM - 1, MAX_DIM]
    rng = random.Random(7)
    ks = [0, 1, 128, 129, 1000, 1 << 16, (1 << 23) - 128, 1 << 23, MAX_DIM]
    sizes = list(itertools.product(edge, edge, ks))
    for _ in range(4000):
        sizes.append(tuple(min(MAX_DIM, int(2 ** rng.uniform(0, 24.001))) for _ in range(3)))
    return [(m, n, k, wide) for m, n, k in sizes if up(m, 128) * up(n, 128) <= MAX_TILES for wide in (0, 1)]


def check_launches(choose):
    sizes = far_sizes()
    assert max(up(m, 128) * up(n, 128) for m, n, _, _ in sizes) > MAX_TILES // 2
    for (m, n, k, wide), c in zip(sizes, choose(sizes)):
        assert c.blocks * 512 < 1 << 32, (m, n, k, wide, c)
        nkb = up(k, 128)
        if c.splits > 1:
            # no split is empty, and the partial sums fit
            assert (c.splits - 1) * c.per < nkb <= c.splits * c.per and c.em == 64
            assert c.ws == 4 * c.splits * m * up(n, 4) * 4
        else:
            assert c.ws == 0 and c.per == nkb
        if c.em >= 128:
            assert nkb * 128 < 1 << 23  # 32-bit offsets within a tile's rows


def test_launches_fit(choose):
    check_launches(choose)


@pytest.mark.parametrize("estimate", ["const double t16 = 0.0;", "const double t16 = 1e-9 * (double)nkb;"])
def test_launches_fit_whatever_the_estimates(tmp_path, estimate):
    src = open(f"{CSRC}/fp8_choice.h").read()
    start = src.index("const double t16 =")
    end = src.index(";", start) + 1
    check_launches(build(tmp_path, src[:start] + estimate + src[end:]))


KERNELS = {"16", "64", "64 split", "128", "192 x 256", "256"}
# what is tested at every kernel, and the GPU tests that do it together
ASPECTS = {
    "values": ["test_product_against_fp64", "test_product_at_every_tile_size_and_loop_length"],
    "adding": ["test_product_of_block_kinds_accumulates", "test_split_products_add_into_strided_rows"],
    "strided": ["test_product_into_strided_rows_writes_nothing_else", "test_split_products_add_into_strided_rows"],
    "nan": ["test_nan_and_overflow_stay_in_their_rows", "test_split_products_keep_nan_in_its_rows"],
    "sums": ["test_sums_are_fp32", "test_split_sums_are_fp32"],
    "ends": ["test_entries_at_the_ends_of_the_range"],
    "fast, ends": ["test_entries_at_the_ends_of_the_range"],
    "fast": ["test_fast_results_keep_their_bound", "test_split_fast_results_keep_their_bound"],
    "fast, strided": ["test_fast_results_added_into_strided_rows"],
}


def kernel(c):
    return {(16, 16): "16", (64, 64): "64 split" if c.splits > 1 else "64", (128, 128): "128", (192, 256): "192 x 256",
            (256, 256): "256"}[c.em, c.en]


def params(test, names):
    """The values that a test is parametrised with under `names`."""
    return next(mark.args[1] for mark in test.pytestmark if mark.name == "parametrize" and mark.args[0] == names)


def sizes_of(test, k=None):
    if k is None:
        return [tuple(s) for s in params(test, "m,n,k")]
    return [(*mn, kk) for mn in params(test, "m,n") for kk in params(test, k)]


@pytest.mark.parametrize("aspect", sorted(ASPECTS))
def test_gpu_tests_reach_every_kernel(choose, aspect):
    sizes = []
    for name in ASPECTS[aspect]:
        fn = next(getattr(m, name) for m in (test_fp8_gpu, test_fp8_sums_gpu, test_fp8_split_gpu, test_fp8_ends_gpu) if hasattr(m, name))
        sizes += sizes_of(fn, "k" if "loop_length" in name else None)
    wide = 0 if "fast" in aspect else 1
    got = {kernel(c) for c in choose([(*s, wide) for s in sizes])}
    assert got == KERNELS
