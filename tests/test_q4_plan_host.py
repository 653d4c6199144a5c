"""The sizes of the products with 4-bit weights, on the host (no GPU)."""

import ctypes
import random
import shutil
import subprocess
from pathlib import Path

import pytest
import torch

from q4_variants import CASES, FAMILIES, FAR, whole

TESTS = Path(__file__).resolve().parent
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    out = tmp_path_factory.mktemp("q4_plan") / "libshim.so"
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", str(TESTS / "q4_plan_shim.cpp"), "-o", str(out)], check=True)
    lib = ctypes.CDLL(str(out))
    lib.shim_staged_bytes.restype = ctypes.c_longlong
    return lib


def test_groups_of_a_row(shim):
    """As many as its columns need, up to an int's end."""
    rng = random.Random(1)
    sizes = [*range(1, 700), *range(MOST - 300, MOST + 1), *(rng.randint(1, MOST) for _ in range(2000))]
    for K in sizes:
        for log2 in range(3):
            assert shim.shim_groups_of(K, log2) == -(-K // (32 << log2)), (K, log2)


def test_the_sizes_that_are_run_reach_every_kernel(shim):
    reached = set()
    for dtype, family, M, K, nvec, pad, shift in CASES:
        parts = 3 if dtype == torch.float32 else 1
        got = FAMILIES[shim.shim_family(parts, M, K, nvec, int(pad >= FAR), int(whole(K, pad, shift)))]
        assert got == family, (dtype, M, K, nvec, pad, shift, got)
        reached.add((dtype, family))
    halves = [f for f in FAMILIES if f != "staged"]
    assert reached == {(t, f) for t in (torch.float16, torch.bfloat16) for f in halves} | {
        (torch.float32, f) for f in FAMILIES if not f.startswith("wide")}


def test_every_kernel_gets_what_it_holds(shim):
    """Vectors that fit LDS, rows that an offset of 32 bits reaches, whole chunks where
    they go straight into LDS, and no more workgroups than a launch has."""
    rows_of = dict(zip(FAMILIES, (256, 16, 16, 32, 64, 64, 128, 256, 256, 256)))
    vectors_of = dict(zip(FAMILIES, (1, 16, 16, 16, 16, 64, 128, 64, 112, 128)))
    threads_of = dict(zip(FAMILIES, (256, 1024, 512, 512, 512, 256, 256, 256, 256, 256)))
    rng = random.Random(2)
    for _ in range(100000):
        parts, far, ok = rng.choice((1, 3)), rng.random() < 0.1, rng.random() < 0.5
        M = min(int(2 ** rng.uniform(0, 20.1)), 1 << 20)
        K, T = min(int(2 ** rng.uniform(0, 31)), MOST), min(int(2 ** rng.uniform(0, 15.1)), 1 << 15)
        family = FAMILIES[shim.shim_family(parts, M, K, T, int(far), int(ok))]
        what = (parts, M, K, T, far, ok, family)
        assert (family == "short") == (K < 32), what
        if family == "staged":
            assert parts == 3 and T <= 5 and shim.shim_staged_bytes(parts, K, T) <= 150 * 1024, what
        if family.startswith(("tile", "wide")):
            assert not far, what
        if family.startswith("wide"):
            assert parts == 1 and ok, what
        rows, vectors = rows_of[family], vectors_of[family]
        if (parts, family) == (3, "tile128"):
            rows, vectors = 192, 64
        across, down = -(-M // rows), -(-T // vectors)
        if family.startswith(("tile", "wide")):
            across, down = across * down, 1
        assert across * threads_of[family] < 1 << 32 and across < 1 << 31 and down <= 65535, what
