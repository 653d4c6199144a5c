"""The mapping of the attention over the paged 8-bit cache, on the host (no
GPU): the chunks that a row tile walks hold every token that its rows see,
once, inside the table; and no row tile has more of them than the launcher
sized the grid, the join and the workspace for."""

import ctypes
import random
import shutil
import subprocess
from pathlib import Path

import pytest

import memory_bound_gemv_f32_amd as lg
from kv_variants import CASES

TESTS = Path(__file__).resolve().parent
CHUNK, MAX_SPLITS, MOST = 64, 512, 2 ** 31 - 1
FIELDS = ("row_tiles", "waves_share", "group_rows", "place_rows", "splits", "split_chunks", "places")


def build_shim(folder) -> ctypes.CDLL:
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    out = folder / "libkv_plan_shim.so"
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", str(TESTS / "kv_plan_shim.cpp"), "-o", str(out)],
                   check=True)
    lib = ctypes.CDLL(str(out))
    lib.shim_span.argtypes = [ctypes.c_int] * 6 + [ctypes.POINTER(ctypes.c_int)]
    lib.shim_span.restype = None
    lib.shim_map.argtypes = [ctypes.c_int] * 6 + [ctypes.c_longlong] + [ctypes.c_int] * 2 + [
        ctypes.POINTER(ctypes.c_longlong)]
    lib.shim_map.restype = None
    lib.shim_workspace.argtypes = lib.shim_map.argtypes
    lib.shim_workspace.restype = None
    return lib


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    return build_shim(tmp_path_factory.mktemp("kv_plan"))


def span(lib, window, sinks, capacity, low, high, length):
    out = (ctypes.c_int * 3)()
    lib.shim_span(window, sinks, capacity, low, high, length, out)
    return tuple(out)


def mapping(lib, q_heads, heads, dim, rows, sequences, one_each, capacity, window=0, sinks=0) -> dict:
    out = (ctypes.c_longlong * 7)()
    lib.shim_map(q_heads, heads, dim, rows, sequences, int(one_each), capacity, window, sinks, out)
    return dict(zip(FIELDS, out))


def chunks_of(first, low, high):
    return list(range(first)) + list(range(low, high))


def test_a_row_tile_walks_what_it_sees_once_and_inside_the_table(shim):
    """Lengths within the table and far past it, tables of no page, windows and
    first tokens of every size."""
    rng = random.Random(1)
    sizes = (0, 1, 5, 63, 64, 65, 130, 1000, 4097)
    for _ in range(40000):
        capacity = rng.choice((0, 16, 64, 100, 256, 1024, 5000)) // 16 * 16
        length = rng.choice((rng.randint(-5, 1200), rng.randint(0, 6000)))
        rows = rng.choice((1, 2, 7, 40))
        high = rng.randint(length - rows, length - 1) if rng.random() < 0.5 else length - 1
        low = max(high - rng.randint(0, rows), length - rows) if rows > 1 else high
        low, window, sinks = min(low, high), rng.choice(sizes), rng.choice(sizes)
        got = span(shim, window, sinks, capacity, low, high, length)
        walked = chunks_of(*got)
        what = (window, sinks, capacity, low, high, length, got)
        assert len(set(walked)) == len(walked) == got[0] + got[2] - got[1], what
        assert len(walked) <= -(-capacity // CHUNK) and all(0 <= c * CHUNK < capacity for c in walked), what
        there = set(walked)
        for p in {low, high}:
            last = min(p, length - 1, capacity - 1)
            seen = range(max(0, p - window + 1) if window else 0, last + 1)
            seen = set(j // CHUNK for j in (seen[::CHUNK] if len(seen) else ())) | ({last // CHUNK} if len(seen) else set())
            if window and last >= 0 and sinks:
                seen |= set(range(0, min(sinks - 1, last) // CHUNK + 1))
            assert seen <= there, what


def test_lengths_up_to_an_int_walk_only_the_table(shim):
    for window, sinks in ((16, MOST), (1, 4000), (MOST, MOST), (70, 0)):
        for capacity in (0, 64, 1024, MOST):
            first, low, high = span(shim, window, sinks, capacity, MOST - 1, MOST - 1, MOST)
            assert 0 <= first <= low <= high <= -(-capacity // CHUNK), (window, sinks, capacity)


def test_no_row_tile_has_more_chunks_than_the_launch(shim):
    """Every tile of random batches, lengths past the table among them: its
    chunks fit the splits, and the splits fit the join."""
    rng = random.Random(2)
    split = 0
    for _ in range(6000):
        heads, group, dim = rng.choice((1, 2, 8)), rng.choice((1, 2, 4, 5, 8, 17, 32, 64)), rng.choice((64, 128, 256))
        sequences = rng.choice((1, 2, 5, 64, 300))
        capacity = rng.choice((0, 1024, 4096, 20000, 131072, 1 << 21)) // 16 * 16
        one = rng.random() < 0.5
        rows = sequences if one else sequences * rng.choice((1, 2, 9, 60, 400))
        window, sinks = rng.choice((0, 1, 16, 500, 5000)), rng.choice((0, 4, 100, 4000, 10 ** 6, MOST))
        m = mapping(shim, heads * group, heads, dim, rows, sequences, one, capacity, window, sinks)
        assert 1 <= m["splits"] <= MAX_SPLITS, m
        if m["splits"] == 1:
            continue
        split += 1
        tile = m["group_rows"] if m["waves_share"] != 1 else 16 * m["row_tiles"]  # rows that a wavefront walks for
        for _ in range(20):
            new = 1 if one else rng.randint(1, max(1, rows // sequences * 2))
            length = rng.choice((rng.randint(1, capacity + 1), capacity, capacity + rng.randint(0, 9 * capacity + 50), MOST))
            r0 = rng.randrange(new * group)
            last = min(r0 + tile, new * group) - 1
            low, high = length - new + r0 // group, length - new + last // group
            first, lo, hi = span(shim, window, sinks, capacity, low, high, length)
            assert first + hi - lo <= m["splits"] * m["split_chunks"], (m, window, sinks, capacity, low, high, length)
    assert split > 500


def test_partial_rows_are_aligned_and_fit_the_workspace(shim):
    """The rows of the workspace start at 16 bytes (they are stored in pieces of
    that), behind every row's maximum and sum, and end with it."""
    rng = random.Random(3)
    odd = 0
    for _ in range(4000):
        heads, group, dim = rng.choice((1, 2, 3)), rng.choice((1, 3, 4, 5)), rng.choice((64, 128, 256))
        sequences, capacity = rng.choice((1, 1, 3, 7)), rng.randrange(0, 1 << 17, 16)
        one = rng.random() < 0.7
        rows = sequences if one else sequences * rng.choice((1, 3, 50))
        args = (heads * group, heads, dim, rows, sequences, one, capacity)
        m = mapping(shim, *args)
        if m["splits"] == 1:
            continue
        out = (ctypes.c_longlong * 2)()
        shim.shim_workspace(*args[:5], int(one), capacity, 0, 0, out)
        parts = m["places"] * heads * m["splits"] * m["place_rows"]
        odd += parts % 2
        assert out[0] % 4 == 0 and out[0] >= 2 * parts, (args, m)
        assert out[1] % 16 == 0 and out[1] == 4 * (out[0] + parts * dim), (args, m)
    assert odd > 20


@pytest.mark.parametrize("name", CASES)
def test_each_mapping_has_its_case(shim, name):
    """The cases that the GPU tests run against the reference have the mapping
    that they are there for (heads of 256 have one row tile and no eight wavefronts)."""
    lens, new, heads, group, page, window, sinks, waves, tiles, split = CASES[name]
    capacity = -(-max(lens) // page) * page
    for dim in (64, 128, 256):
        rows = len(lens) if new is None else sum(new)
        m = mapping(shim, heads * group, heads, dim, rows, len(lens), new is None, capacity, window, sinks)
        if dim == 256:
            assert m["row_tiles"] == 1 and m["waves_share"] == (1 if waves == 1 else 4), m
        else:
            assert (m["waves_share"], m["row_tiles"], m["splits"] > 1) == (waves, tiles, split), m


def test_sizes_that_one_launch_always_holds():
    """sequences x heads up to 2^22 and rows x q_heads up to 2^29, as documented."""
    rng = random.Random(4)
    n = ctypes.c_size_t()
    for _ in range(20000):
        heads = rng.choice((1, 2, 3, 8, 64, 1000, 65535))
        sequences = rng.choice((1, 7, (1 << 22) // heads, rng.randint(1, (1 << 22) // heads)))
        group = rng.choice((1, 2, 4, 8, 16, 17, 32, 33, 64, 128, 1000))
        most = (1 << 29) // (heads * group)
        one = rng.random() < 0.3 and sequences <= most
        if most < 1:
            continue
        rows = sequences if one else rng.choice((1, most, rng.randint(1, most), min(most, sequences * rng.choice((1, 16, 17, 32, 33)))))
        rc = lg.gemv_kv_attend_workspace_size(heads * group, heads, rng.choice((64, 128, 256)), rows, sequences, int(one),
                                              rng.choice((1, 100, 1 << 20, MOST)), rng.choice((16, 256)),
                                              rng.choice((0, 0, 1000)), rng.choice((0, 70)), ctypes.byref(n))
        assert rc == 0, (heads, group, rows, sequences, one)
