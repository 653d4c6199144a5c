"""The sizes of the products with 4-bit weights, on the host (no GPU)."""

import ctypes
import random
import shutil
import subprocess
from pathlib import Path

import pytest

TESTS = Path(__file__).resolve().parent
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    out = tmp_path_factory.mktemp("q4_plan") / "libshim.so"
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", str(TESTS / "q4_plan_shim.cpp"), "-o", str(out)], check=True)
    return ctypes.CDLL(str(out))


def test_groups_of_a_row(shim):
    """As many as its columns need, up to an int's end."""
    rng = random.Random(1)
    sizes = [*range(1, 700), *range(MOST - 300, MOST + 1), *(rng.randint(1, MOST) for _ in range(2000))]
    for K in sizes:
        for log2 in range(3):
            assert shim.shim_groups_of(K, log2) == -(-K // (32 << log2)), (K, log2)
