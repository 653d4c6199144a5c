"""Every mapping of the attention over the paged 8-bit cache, and batches of
many sequences, against the reference in 64 bits (needs a GPU)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import memory_bound_gemv_f32_amd as lg
from fp8_helpers import Batch, PlainCache
from kv_variants import CASES
from test_kv_gpu import BF16, E4M3, F16, F32, INT8, assert_same_cache, check_attend, f64, filled, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("form,dtype", [(INT8, BF16), (E4M3, F16), (INT8, F16), (E4M3, BF16)])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("name", CASES)
def test_attend(name, dim, form, dtype):
    lens, new, heads, group, page, window, sinks, waves, tiles, split = CASES[name]
    batch = Batch(lens, [1] * len(lens) if new is None else new, page, np.random.default_rng(dim))
    check_attend(batch, heads, group, dim, page, form, dtype, window=window, sinks=sinks, one_each=new is None, seed=dim)


@pytest.mark.parametrize("form", [INT8, E4M3])
@pytest.mark.parametrize("many", [65, 130, 300])
def test_append_to_many_sequences(many, form):
    """Batches whose sequences are searched for, some of them without new tokens."""
    rng = np.random.default_rng(many)
    new = [int(n) for n in rng.choice((0, 0, 1, 2, 17, 40), many)]
    lens = [n + int(rng.integers(0, 60)) for n in new]
    heads, dim, page = 1, 64, 32
    batch = Batch(lens, new, page, rng)
    cache = filled(batch.pages, heads, dim, page, form, many)
    plain = PlainCache(cache)
    K, V = values(1, batch.rows, heads, dim, F32, 3.0), values(2, batch.rows, heads, dim, F32, 0.05)
    lg.gemv_kv_append(cache, K, V, *batch.tensors())
    plain.append(f64(K), f64(V), batch)
    assert_same_cache(cache, plain)


def test_captured_split_calls_replay():
    """Two captured calls that take a workspace, of single tokens and of a
    prompt's chunk behind padding rows, replayed in turn while the lengths in
    device memory grow and eager calls run between: every replay equals the
    eager call."""
    rng = np.random.default_rng(1)
    calls = []
    for lens, new, pad, window in (([2000, 700], None, 0, 0), ([3000, 90], [70, 9], 5, 1500)):
        batch = Batch([n + 400 for n in lens], [1] * 2 if new is None else new, 64, rng)
        cache = filled(batch.pages, 2, 128, 64, E4M3, 1)
        table, length, starts = batch.tensors(new is not None)
        length.copy_(torch.tensor(lens, dtype=torch.int32))
        Q = values(1, batch.rows + pad, 8, 128, BF16)
        need = lg.kv_attend_workspace_size(cache, 8, len(Q), 2, table.shape[1], one_each=new is None, window=window, sinks=4)
        assert need > 0
        def call(out, args=(Q, cache, table, length, starts), window=window):
            return lg.gemv_kv_attend(*args, window=window, sinks=4, out=out)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        out = torch.full_like(Q, 3.0)
        with torch.cuda.stream(side):
            call(out)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(out)
        calls.append((graph, call, out, Q, length, lens))
    for step in range(12):
        for graph, call, out, Q, length, lens in calls:
            length.copy_(torch.tensor([n + 33 * step for n in lens], dtype=torch.int32))
            Q.copy_(torch.roll(Q, 1, 0))
        for graph, *_ in calls:
            graph.replay()
        for graph, call, out, Q, length, lens in calls:
            want = call(torch.full_like(Q, 3.0))
            assert torch.equal(out, want) and torch.isfinite(want).all(), step
        if step % 4 == 0:
            torch.cuda.synchronize()
