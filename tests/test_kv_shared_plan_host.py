"""The mapping of the attention behind shared tokens, on the host (no GPU): the
shared chunks and a row tile's own ones are together what it sees, once; both
parts' splits hold all of their chunks; and the workspace holds both parts."""

import ctypes
import random
import shutil
import subprocess
from pathlib import Path

import pytest

import memory_bound_gemv_f32_amd as lg

TESTS = Path(__file__).resolve().parent
CHUNK = 64
FIELDS = ("row_tiles", "waves_share", "group_rows", "place_rows", "splits", "split_chunks", "places")


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    out = tmp_path_factory.mktemp("kv_shared_plan") / "libshim.so"
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", str(TESTS / "kv_shared_plan_shim.cpp"), "-o", str(out)],
                   check=True)
    lib = ctypes.CDLL(str(out))
    lib.shim_span_from.argtypes = [ctypes.c_int] * 7 + [ctypes.POINTER(ctypes.c_int)]
    lib.shim_map_both.argtypes = [ctypes.c_int] * 6 + [ctypes.c_longlong] + [ctypes.c_int] * 3 + [
        ctypes.POINTER(ctypes.c_longlong)]
    return lib


def walked(lib, window, sinks, capacity, low, high, length, begin):
    out = (ctypes.c_int * 4)()
    lib.shim_span_from(window, sinks, capacity, low, high, length, begin, out)
    return [lib.shim_chunk_from(*out, i) for i in range(lib.shim_count_from(*out))]


def test_own_chunks_are_those_behind_the_shared(shim):
    rng = random.Random(1)
    sizes = (0, 1, 5, 63, 64, 65, 130, 1000, 4097)
    for _ in range(40000):
        capacity = rng.choice((0, 16, 64, 100, 256, 1024, 5000)) // 16 * 16
        length = rng.choice((rng.randint(-5, 1200), rng.randint(0, 6000)))
        high = length - 1 - rng.choice((0, 0, rng.randint(0, 50)))
        low, window, sinks = high - rng.randint(0, 30), rng.choice(sizes), rng.choice(sizes)
        begin = rng.choice((0, 1, 2, 7, rng.randint(0, 90)))
        every = walked(shim, window, sinks, capacity, low, high, length, 0)
        assert walked(shim, window, sinks, capacity, low, high, length, begin) == [c for c in every if c >= begin], (
            window, sinks, capacity, low, high, length, begin)


def mapping(lib, *args):
    out = (ctypes.c_longlong * 19)()
    lib.shim_map_both(*args, out)
    out = list(out)
    return out[0], dict(zip(FIELDS, out[1:8])), dict(zip(FIELDS, out[8:15])), *out[15:]


def drawn(rng):
    heads = rng.choice((1, 2, 5, 8, 32))
    group, dim = rng.choice((1, 2, 4, 5, 7, 8, 16, 17, 32, 40)), rng.choice((64, 128, 256))
    sequences, one_each = rng.choice((1, 2, 3, 4, 8, 9, 16, 64, 300)), rng.random() < 0.5
    rows = sequences if one_each else rng.choice((sequences, rng.randint(1, 40 * sequences), 5 * sequences))
    shared = rng.choice((0, 1, 63, 64, 500, rng.randint(1, 4000), rng.randint(1, 100000), 2 ** 31 - 1))
    capacity = rng.choice((0, 16, 128, 600, rng.randint(1, 5000), min(2 ** 31 - 1, shared + 1000), 200000)) // 16 * 16
    window = rng.choice((0, 0, 0, 1, 100, 5000, 100000))
    return heads * group, heads, dim, rows, sequences, int(one_each), capacity, window, rng.choice((0, 4, 70, 5000)), shared


def test_both_parts_are_whole_and_the_workspace_holds_them(shim):
    rng = random.Random(2)
    parts = fused = 0
    for _ in range(40000):
        args = drawn(rng)
        q_heads, heads, dim, rows, sequences, one_each, capacity, window, sinks, shared = args
        chunks, prefix, own, together, launchable, bytes_all, bytes_prefix = mapping(shim, *args)
        assert launchable, args
        assert chunks * CHUNK <= min(shared, capacity) and chunks * CHUNK > min(shared, capacity) - CHUNK or chunks == 0, args
        if chunks == 0:
            continue
        parts += 1
        fused += together
        all_rows = rows * (q_heads // heads)
        assert prefix["waves_share"] == 4 and prefix["group_rows"] == 16 * prefix["row_tiles"], args
        assert prefix["places"] * prefix["group_rows"] >= all_rows, args
        assert (prefix["places"] - 1) * prefix["group_rows"] < all_rows, args
        assert prefix["place_rows"] == min(all_rows, prefix["group_rows"]), args
        assert prefix["splits"] * prefix["split_chunks"] >= chunks, args
        assert prefix["splits"] <= 512 and own["splits"] <= 512, args
        if own["splits"] > 1:  # (a single split takes what there is)
            tokens = -(-own["group_rows"] // (q_heads // heads)) + 1
            for _ in range(4):
                high = rng.choice((capacity - 1, rng.randint(0, capacity + 100)))
                low = max(high - rng.randint(0, tokens - 1), 0)
                count = len(walked(shim, window, sinks, capacity, low, high, high + 1, chunks)) if high < 10000 else 0
                assert count <= own["splits"] * own["split_chunks"], (args, low, high)
        if together:
            assert own["waves_share"] == 4 and own["row_tiles"] == 1, args
        # every workgroup's rows, their maxima and sums, in floats
        need = 0
        for m in (prefix, own):
            n = m["places"] * heads * m["splits"] * m["place_rows"]
            need += 4 * (-(-2 * n // 4) * 4 + n * dim)
        assert bytes_all == need and bytes_prefix % 16 == 0 and bytes_prefix < need, args
    assert parts > 3000 and fused > 1000


def test_the_library_reports_the_same_workspace(shim):
    """The entry point reports what the mapping needs."""
    rng = random.Random(3)
    for _ in range(200):
        args = drawn(rng)
        q_heads, heads, dim, rows, sequences, one_each, capacity, window, sinks, shared = args
        n = ctypes.c_size_t()
        assert lg.gemv_kv_attend_shared_workspace_size(q_heads, heads, dim, rows, sequences, one_each, capacity // 16, 16,
                                                       window, sinks, shared, ctypes.byref(n)) == 0
        assert n.value == mapping(shim, *args)[5], args


def test_sharing_where_it_pays(shim):
    """Single tokens from 16 MiB of keys over all sequences on, prompts of few
    sequences not."""
    def chunks(sequences, shared, rows=None, heads=8, dim=128, window=0, sinks=0):
        rows = sequences if rows is None else rows
        return mapping(shim, 4 * heads, heads, dim, rows, sequences, int(rows == sequences), shared + 1024, window, sinks,
                       shared)[0]
    assert chunks(4, 4096) == 64 and chunks(4, 4032) == 0
    assert chunks(64, 256) == 4 and chunks(1, 1 << 20) == 0 and chunks(300, 63) == 0
    assert chunks(4, 8192, 200) == 0 and chunks(12, 4000, 1000) == 62
    # windows that hide a part
    assert chunks(64, 4096, window=2048) == 64 and chunks(64, 4096, window=2047) == 0
    assert chunks(64, 4096, window=2000, sinks=48) == 64 and chunks(4, 4096, window=5000) == 64


def test_prompts_that_fill_the_gpu_are_not_taken_together(shim):
    """Behind few shared tokens they take longer together (measured beside the rule);
    behind many, or with few rows each, they do not."""
    def chunks(sequences, new, shared, group=4, heads=8, dim=128):
        return mapping(shim, group * heads, heads, dim, sequences * new, sequences, 0, shared + new + 64, 0, 0, shared)[0]
    for sequences, new, shared, group in ((16, 1000, 4096, 4), (64, 512, 1024, 1), (12, 150, 4096, 4), (64, 128, 4096, 4),
                                          (256, 48, 1024, 1), (1000, 34, 512, 1), (16, 100, 2048, 4)):
        assert chunks(sequences, new, shared, group) == 0, (sequences, new, shared, group)
    for sequences, new, shared, group in ((12, 80, 4096, 4), (16, 1000, 16384, 4), (256, 48, 4096, 1), (64, 49, 4096, 2),
                                          (16, 100, 2048, 1), (16, 256, 4096, 1)):
        assert chunks(sequences, new, shared, group) == shared // 64, (sequences, new, shared, group)


def workspace(q_heads, heads, dim, rows, sequences, one_each, width, page, window, sinks, shared):
    """Bytes of a call with and without shared tokens; None where it is refused."""
    out = []
    for n in (shared, 0):
        size = ctypes.c_size_t()
        status = lg.gemv_kv_attend_shared_workspace_size(q_heads, heads, dim, rows, sequences, one_each, width, page, window,
                                                         sinks, n, ctypes.byref(size))
        out.append(size.value if status == 0 else None)
    return out


def test_the_workspace_is_bounded():
    """However many rows, heads and sequences there are: 1 GiB, or what the call needs
    without shared tokens."""
    for args in ((32, 8, 128, 64000, 32, 0, 1024, 64, 0, 0, 16384), (32, 8, 128, 128000, 64, 0, 300, 64, 0, 0, 16384),
                 (1, 1, 64, 1 << 22, 1 << 17, 0, 2000, 64, 0, 0, 100000), (64, 1, 256, 1 << 18, 1 << 18, 1, 5000, 64, 0, 0, 300000),
                 (128, 128, 256, 100000, 3000, 0, 5000, 64, 0, 0, 300000)):
        with_shared, without = workspace(*args)
        assert without is not None and with_shared <= max(1 << 30, without), args
    rng = random.Random(6)
    for _ in range(20000):
        heads, group = rng.choice((1, 2, 8, 32, 128)), rng.choice((1, 2, 4, 8, 16, 40))
        sequences = int(2 ** rng.uniform(1, 18))
        rows = sequences * int(2 ** rng.uniform(0, 11))
        if rows * heads * group >= 1 << 31:
            continue
        with_shared, without = workspace(heads * group, heads, rng.choice((64, 128, 256)), rows, sequences,
                                         int(rows == sequences and rng.random() < 0.5), int(2 ** rng.uniform(0, 16)), 64,
                                         rng.choice((0, 0, 5000)), 0, int(2 ** rng.uniform(6, 22)))
        assert with_shared is None or with_shared <= max(1 << 30, without)
        assert (with_shared is None) == (without is None)


def test_no_call_is_refused_for_its_shared_tokens():
    """Up to the sizes that the call takes without them."""
    for dim in (64, 128, 256):
        for log2 in (28, 29):
            for sequences in (8, 1 << 16, 1 << 20):
                for q_heads, heads in ((1, 1), (32, 8), (64, 64)):
                    if sequences * heads > 1 << 22:
                        continue
                    rows = (1 << log2) // q_heads
                    if rows < sequences:
                        continue
                    with_shared, without = workspace(q_heads, heads, dim, rows, sequences, 0, 1 << 20, 64, 0, 0, 1 << 20)
                    assert with_shared is not None and without is not None, (dim, log2, sequences, q_heads, heads)


def test_no_launch_is_larger_than_the_runtime_takes(shim):
    """Where the parts are launched the join is too: a thread of every tile's
    workgroup is counted in 32 bits."""
    for rows in (1000, 30000, 65500, 120000):
        for dim in (64, 128, 256):
            for heads in (8, 4096, 8192, 32768):
                args = (heads, heads, dim, rows, rows // 33, 0, 1 << 20, 0, 0, 1 << 16)
                chunks, prefix, own, _, launchable, *_ = mapping(shim, *args)
                assert chunks > 0
                if launchable:
                    assert own["places"] * heads * 256 < 1 << 32, args
                    assert prefix["places"] * heads * prefix["splits"] * 256 < 1 << 32, args
