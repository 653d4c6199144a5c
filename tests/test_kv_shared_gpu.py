"""Attention for a batch whose sequences share their first tokens, against the
reference in 64 bits and the call without ``shared`` (needs a GPU)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import memory_bound_gemv_f32_amd as lg
from fp8_helpers import Batch, PlainCache, assert_close, attend
from test_kv_gpu import E4M3, INT8, f64, filled, values

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def shared_problem(lens, new, shared, page_size, heads, dim, form, seed=0, padding=0):
    """A batch whose tables name the same pages for whole shared ones, and copies
    of the first row's where a page is shared in part; the first row has pages for
    all shared tokens, whatever its length."""
    rng = np.random.default_rng(seed)
    first = max(lens[0], shared)
    batch = Batch([first] + list(lens[1:]), new, page_size, rng)
    batch.lens[0] = lens[0]
    cache = filled(batch.pages, heads, dim, page_size, form, seed)
    whole = shared // page_size
    for b in range(1, len(lens)):
        for i in range(-(-min(shared, lens[b]) // page_size)):
            mine, its = int(batch.table[b, i]), int(batch.table[0, i])
            if i < whole:
                batch.table[b, i] = its
            else:
                for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
                    t.view(torch.uint8)[mine] = t.view(torch.uint8)[its]
    batch.rows += padding
    return batch, cache


def check(lens, new, shared, page_size=64, heads=2, group=4, dim=128, form=INT8, dtype=BF16, window=0, sinks=0, seed=0,
          one_each=None, padding=0, scale=None):
    batch, cache = shared_problem(lens, new, shared, page_size, heads, dim, form, seed, padding)
    plain = PlainCache(cache)
    Q = values(seed + 7, batch.rows, heads * group, dim, dtype, 0.2)
    one_each = all(m == 1 for m in new) and not padding if one_each is None else one_each
    tensors = batch.tensors(not one_each)
    out = torch.full_like(Q, 3.0)
    got = lg.gemv_kv_attend(Q, cache, *tensors, window=window, sinks=sinks, shared=shared, out=out, scale=scale)
    assert got is out
    what = f"{lens} {new} shared {shared} page {page_size} {heads}x{group} dim {dim} {form} {dtype} window {window} {sinks}"
    n = int(batch.starts[-1])
    want, bound = attend(f64(Q), plain, batch, dim ** -0.5 if scale is None else scale, window, sinks, dtype)
    assert_close(got[:n], want[:n], bound[:n], what)
    assert (out[n:] == 3.0).all()
    return batch, cache, Q, tensors


@pytest.mark.parametrize("form", [INT8, E4M3])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_one_token_each(dim, dtype, form):
    for n, (lens, shared) in enumerate([([100, 90], 64), ([200, 150, 130], 127), ([700, 650, 641, 655], 640),
                                        ([300] * 9, 256), ([1000, 400, 999], 330), ([65, 65], 65)]):
        check(lens, [1] * len(lens), shared, [16, 32, 64, 128, 256][n % 5], 1 + n % 2, [1, 4, 5, 8, 3, 16][n], dim, form, dtype, seed=n)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("form", [INT8, E4M3])
def test_prompts(dim, form):
    for n, (lens, new, shared) in enumerate([([200, 150], [20, 3], 128), ([400, 390, 330, 385], [70, 1, 8, 64], 300),
                                             ([150, 150, 150], [5, 0, 22], 100), ([300] * 6, [40] * 6, 256)]):
        check(lens, new, shared, [32, 16, 64, 128][n], 2, [4, 2, 8, 1][n], dim, form, F16, seed=n)


@pytest.mark.parametrize("rows", [2, 5, 9, 17, 33, 64, 70])
def test_rows(rows):
    """Row tiles of every kind, full and not."""
    for group in (1, 4, 7):
        check([260 + 7 * (i % 5) for i in range(rows)], [1] * rows, 256, 64, 1, group, 128, INT8, BF16, seed=rows)


def test_long_shared():
    """Several splits of the shared tokens and of the own ones."""
    check([5000, 4500, 4100], [1, 1, 1], 4096, 128, 1, 4, 128, E4M3, BF16)
    check([9000, 8300], [3, 1], 8192, 256, 1, 2, 64, INT8, F16)
    check([4000, 3900, 3999, 3950], [30, 20, 10, 40], 3900, 16, 1, 2, 128, INT8, F16)


def test_windows():
    """Windows that see all, a part or nothing of the shared tokens, with and
    without first tokens that stay visible."""
    for n, (window, sinks) in enumerate([(16, 0), (16, 4), (64, 70), (200, 0), (300, 1), (10000, 4), (500, 1000), (1, 0)]):
        for lens, new in (([400, 330, 500], [1, 1, 1]), ([400, 330, 500], [30, 20, 90])):
            check(lens, new, 320, [16, 64][n % 2], 2, 3, 128, [INT8, E4M3][n % 2], BF16, window, sinks, seed=n)


def test_rows_inside_the_shared_tokens():
    """Sequences that end within the shared tokens see their own part of them."""
    check([300, 40, 1, 200], [1, 1, 1, 1], 256, 64)
    check([300, 64, 70, 200, 256], [20, 64, 6, 150, 1], 256, 32)
    check([0, 300, 280], [0, 4, 2], 256, 64)                # an empty first sequence, whose pages are there
    check([0, 300, 280], [0, 4, 2], 256, 64, window=100, sinks=5)


def test_padding_rows_stay():
    check([300, 290], [4, 3], 256, 64, padding=9)
    check([300, 290], [1, 1], 256, 64, padding=30)


def test_negative_and_zero_scale():
    check([300, 290, 270], [1, 1, 1], 256, 64, scale=-0.05)
    check([300, 290, 270], [1, 1, 1], 256, 64, scale=0.0)


def test_missing_pages():
    """Shared tokens whose page is not there are not seen."""
    batch, cache = shared_problem([400, 390, 350], [1, 1, 1], 320, 32, 2, 128, INT8)
    for bad in (-1, batch.pages, 1 << 30):
        batch.table[:, 3] = bad
        Q = values(1, 3, 8, 128, BF16)
        got = lg.gemv_kv_attend(Q, cache, *batch.tensors(False), shared=320)
        assert_close(got, *attend(f64(Q), PlainCache(cache), batch, 128 ** -0.5, dtype=BF16))


def test_more_shared_than_the_table_holds():
    batch, cache = shared_problem([256, 256], [1, 1], 256, 64, 2, 128, INT8)
    Q = values(1, 2, 8, 128, BF16)
    got = lg.gemv_kv_attend(Q, cache, *batch.tensors(False), shared=1 << 30)
    assert_close(got, *attend(f64(Q), PlainCache(cache), batch, 128 ** -0.5, dtype=BF16))


def test_hidden_blocks_that_are_not_finite():
    """A NaN scale reaches the rows that see its block, and no others."""
    batch, cache = shared_problem([400, 150, 390], [1, 1, 1], 384, 64, 1, 128, E4M3)
    page = int(batch.table[0, 3])
    cache.k_scale[page, 0, 1] = float("nan")        # tokens 208 to 223
    Q = values(2, 3, 4, 128, F16)
    got = lg.gemv_kv_attend(Q, cache, *batch.tensors(False), shared=384)
    assert torch.isnan(got[0]).all() and torch.isnan(got[2]).all()
    want, bound = attend(f64(Q), PlainCache(cache), batch, 128 ** -0.5, dtype=F16)
    assert_close(got[1], want[1], bound[1])
    cache.k_scale[page, 0, 1] = 1.0
    hidden = PlainCache(cache)  # (the window of 100 hides the block: its V scale has no part in the bound)
    cache.v_scale[page, 0, 1] = float("inf")
    got = lg.gemv_kv_attend(Q, cache, *batch.tensors(False), shared=384, window=100)
    assert_close(got, *attend(f64(Q), hidden, batch, 128 ** -0.5, 100, 0, dtype=F16))


def test_a_row_does_not_depend_on_the_others():
    """A row's bits are the same whatever the other rows hold, and from call to
    call."""
    batch, cache, Q, tensors = check([700, 650, 660, 690], [1, 1, 1, 1], 640, heads=1)
    first = lg.gemv_kv_attend(Q, cache, *tensors, shared=640)
    assert torch.equal(first, lg.gemv_kv_attend(Q, cache, *tensors, shared=640))
    other = Q.clone()
    other[1:] *= 30
    assert torch.equal(first[0], lg.gemv_kv_attend(other, cache, *tensors, shared=640)[0])
    other[1:] = float("nan")
    assert torch.equal(first[0], lg.gemv_kv_attend(other, cache, *tensors, shared=640)[0])


def test_workspace_and_graph():
    batch, cache, Q, tensors = check([700, 650, 660, 690], [1, 1, 1, 1], 640, heads=2)
    width = batch.table.shape[1]
    need = lg.kv_attend_workspace_size(cache, 8, 4, 4, width, shared=640)
    assert need > 0
    guard = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")
    want = lg.gemv_kv_attend(Q, cache, *tensors, shared=640)
    got = lg.gemv_kv_attend(Q, cache, *tensors, shared=640, workspace=guard[:need])
    assert torch.equal(got, want) and (guard[need:] == 77).all()
    with pytest.raises(lg.GemvError):
        lg.gemv_kv_attend(Q, cache, *tensors, shared=640, workspace=guard[:need - 16])
    out = torch.empty_like(Q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lg.gemv_kv_attend(Q, cache, *tensors, shared=640, out=out, workspace=guard[:need])
    for n in range(3):
        Q.copy_(values(n, 4, 8, 128, BF16))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, lg.gemv_kv_attend(Q, cache, *tensors, shared=640)), n


def test_a_step_of_a_model():
    """A decode step and a prompt step as they are used: 4-bit products, norms and
    rotary positions, the append and the attention behind a shared prefix, against
    the same in 64 bits with the library's roundings between the operators."""
    from q4_helpers import product, rotary
    heads, group, dim, hidden, page, prefix = 2, 4, 64, 256, 16, 200
    g = torch.Generator().manual_seed(3)
    width = (heads * group + 2 * heads) * dim
    W = torch.randint(0, 256, (width, hidden // 2), generator=g, dtype=torch.uint8).cuda()
    scale = (torch.rand(width, hidden // 32, generator=g) * 0.01).cuda()
    frequency, magnitude = lg.rotary_frequencies(dim, 10000.0, factor=2.0, original=128)
    weight = [(1 + 0.1 * torch.randn(dim, generator=g)).cuda() for _ in range(2)]
    lens, new = [prefix + 30, prefix + 9, prefix + 20], [1, 1, 1]
    for prompt in (False, True):
        if prompt:
            new = [20, 1, 9]
        batch, cache = shared_problem(lens, new, prefix, page, heads, dim, INT8, seed=4)
        table, seq_lens, starts = batch.tensors(prompt)
        x = torch.randn(batch.rows, hidden, generator=g).cuda()
        qkv = lg.gemv_q4(W, scale, x, group=32)
        assert_close(qkv, *product(W, scale, x, None, None, 32, F32))
        qkv = qkv.view(-1, heads * group + 2 * heads, dim)
        Q, K, V = qkv.split((heads * group, heads, heads), dim=1)
        Qr, Kr = lg.gemv_rotary(Q, K, frequency, seq_lens, starts, q_weight=weight[0], k_weight=weight[1],
                                magnitude=magnitude, q_dtype=F16)
        at = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)])
        assert_close(Qr, *rotary(Q, at, frequency, weight[0], 1e-6, magnitude, False, F16))
        assert_close(Kr, *rotary(K, at, frequency, weight[1], 1e-6, magnitude, False, F32))
        plain = PlainCache(cache)
        plain.append(f64(Kr), f64(V), batch)
        lg.gemv_kv_append(cache, Kr, V, table, seq_lens, starts)
        got = lg.gemv_kv_attend(Qr, cache, table, seq_lens, starts, shared=prefix)
        assert_close(got, *attend(f64(Qr), plain, batch, dim ** -0.5, dtype=F16))
