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


def taken_together(cache, q_heads, rows, sequences, width, one_each, shared, window=0, sinks=0):
    """Whether the library takes the shared tokens for all rows together: then its
    workspace is not the one without them, at one width of the table or another
    (the two can be alike at one by chance)."""
    def size(width, n):
        return lg.kv_attend_workspace_size(cache, q_heads, rows, sequences, width, one_each=one_each, window=window,
                                           sinks=sinks, shared=n)
    return any(size(w, shared) != size(w, 0) for w in (width, width + 3, 2 * width, 8 * width))


def enough_heads(sequences, shared, dim):
    """Key/value heads with which sharing is worth while for single tokens."""
    heads = 1
    while sequences * shared * dim * heads < 1 << 24:
        heads *= 2
    return heads


def check(lens, new, shared, page_size=64, heads=None, group=1, dim=128, form=INT8, dtype=BF16, window=0, sinks=0, seed=0,
          one_each=None, padding=0, scale=None, together=True):
    heads = enough_heads(len(lens), shared, dim) if heads is None else heads
    batch, cache = shared_problem(lens, new, shared, page_size, heads, dim, form, seed, padding)
    plain = PlainCache(cache)
    Q = values(seed + 7, batch.rows, heads * group, dim, dtype, 0.2)
    one_each = all(m == 1 for m in new) and not padding if one_each is None else one_each
    assert together == taken_together(cache, heads * group, batch.rows, len(lens), batch.table.shape[1], one_each, shared,
                                      window, sinks)
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
    """Every head size, type and page size; shared tokens that end inside a page, a
    block and a chunk; row tiles of 16 and of 32 for the batch."""
    for n, (lens, shared, group) in enumerate([([700, 650, 641, 655], 640, 1), ([600] * 9, 513, 1), ([1000, 990, 999, 1001], 983, 5),
                                               ([513, 600, 513, 700, 520, 600], 512, 4), ([530] * 20, 527, 1)]):
        check(lens, [1] * len(lens), shared, [16, 32, 64, 128, 256][n], group=group, dim=dim, form=form, dtype=dtype, seed=n)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [17, 32, 40])
def test_wide_groups(dim, group):
    """Query heads of one key/value head that fill one row tile or several by
    themselves: the own tokens go to other kernels."""
    sequences = 64 if group > 32 else 8
    check([540 + n % 7 for n in range(sequences)], [1] * sequences, 512, 64, group=group, dim=dim, form=E4M3, dtype=F16,
          heads=2 if group > 32 else 16, together=sequences * 512 * dim * 16 >= 1 << 24 or group > 32)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("form", [INT8, E4M3])
def test_few_new_tokens(dim, form):
    for n, (new, group) in enumerate([([1, 3, 2, 1, 4, 1, 2, 5], 2), ([1, 0, 3, 1, 2, 2, 1, 0, 7], 4), ([2] * 12, 1)]):
        lens = [600 + (5 * b) % 60 for b in range(len(new))]
        check(lens, new, 580, [32, 16, 128][n], group=group, dim=dim, form=form, dtype=F16, seed=n)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompts(dim):
    """Prompts of many sequences, whose own rows fill their tiles."""
    rng = np.random.default_rng(dim)
    new = [int(x) for x in rng.integers(10, 40, 64)]
    lens = [512 + m + int(x) for m, x in zip(new, rng.integers(0, 90, 64))]
    check(lens, new, 512, 64, heads=1, group=2, dim=dim, form=E4M3, dtype=BF16)
    check([4100 + 30 * b for b in range(9)], [30, 1, 9, 0, 40, 22, 30, 17, 40], 4096, 128, heads=2, group=2, dim=dim, form=INT8,
          dtype=F16, window=[0, 1000, 4000][dim // 128], sinks=5, together=dim == 64)


@pytest.mark.parametrize("rows", [4, 5, 9, 17, 33, 64, 70])
def test_rows(rows):
    """Row tiles of every kind, full and not."""
    for group in (1, 4, 7):
        check([560 + 7 * (i % 5) for i in range(rows)], [1] * rows, 512, 64, group=group, seed=rows)


def test_long_shared():
    """Several splits of the shared tokens, few and many, and of the own ones."""
    check([5000, 4500, 4100, 4200], [1, 1, 1, 1], 4096, 128, 8, 4, 128, E4M3, BF16)
    check([9000, 8300], [1, 1], 8192, 256, 16, 2, 64, INT8, F16)
    check([70000, 66000], [1, 1], 65536, 256, 2, 2, 64, INT8, F16)
    check([14000, 33000, 33010, 33100], [1, 1, 1, 1], 13000, 64, 4, 2, 128, INT8, F16)
    check([2600 + n for n in range(80)], [1] * 80, 2500, 16, 8, 8, 64, INT8, F16)


def test_windows():
    """Windows that see all, a part or nothing of the shared tokens, with and
    without first tokens that stay visible."""
    for n, (window, sinks) in enumerate([(16, 0), (16, 4), (64, 70), (200, 0), (500, 1), (10000, 4), (700, 1000), (1, 0)]):
        for lens, new in (([900, 830, 1000, 890], [1] * 4), ([900, 830, 1000, 890] * 2, [3, 2, 9, 1] * 2)):
            check(lens, new, 820, [16, 64][n % 2], group=2, form=[INT8, E4M3][n % 2], window=window, sinks=sinks, seed=n,
                  together=window + sinks >= 820)


@pytest.mark.parametrize("new,window,sinks,form", [([1] * 16, 1100, 0, INT8), ([3, 2, 9, 1] * 4, 1024, 5, E4M3),
                                                   ([3, 2, 9, 1] * 4, 1400, 70, INT8), ([1] * 16, 90, 1300, E4M3)])
def test_windows_over_much(new, window, sinks, form):
    """Windows that hide a part of many shared tokens, and leave enough of them to
    take together; a first sequence shorter than the window."""
    lens = [40 if max(new) == 1 else 1900, 1510, 1760, 1530, 1600, 1501, 2700, 1640] + [1900, 1510, 700, 1530] * 2
    check(lens, new, 1500, 64, heads=64, form=form, window=window, sinks=sinks)


def test_windows_of_prompts():
    check([4510 + 7 * b for b in range(64)], [b % 10 + 15 for b in range(64)], 4500, 64, heads=1, group=2, dim=64, form=E4M3,
          window=4200, sinks=5)


def test_rows_inside_the_shared_tokens():
    """Sequences that end within the shared tokens see their own part of them."""
    check([600, 40, 1, 500], [1, 1, 1, 1], 512, 64)
    check([600, 64, 70, 400, 512, 300, 514, 10], [4, 6, 1, 3, 1, 0, 2, 10], 512, 32)
    check([0, 600, 580, 590, 600, 601, 602, 603], [0, 4, 2, 1, 1, 1, 1, 1], 512, 64)  # an empty first sequence, whose pages are there
    check([0, 600, 580, 590, 600, 601, 602, 603], [0, 4, 2, 1, 1, 1, 1, 1], 512, 64, window=200, sinks=5, together=False)


@pytest.mark.parametrize("form", [INT8, E4M3])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_that_see_nothing(dim, form):
    """Empty slots of a batch, the first among them, and rows in front of their
    sequence's first token give exactly 0, beside rows that see every shared token;
    row tiles of 16 and of 32, and prompts."""
    for n, (lens, new, group) in enumerate([
            ([600, 0, 590, 580], [1] * 4, 1), ([0, 600, 0, 590], [1] * 4, 5), ([0] * 3 + [600] * 17, [1] * 20, 2),
            ([600, 3, 590, 0, 700, 650, 1, 680], [2, 5, 1, 2, 1, 3, 4, 1], 2),
            ([0, 600, 590, 580, 570, 0, 700, 650], [1, 6, 1, 2, 1, 3, 4, 1], 4)]):
        check(lens, new, 513 + n, [16, 32, 64, 128, 256][n], group=group, dim=dim, form=form, dtype=[F16, BF16][n % 2], seed=n)
    lens, new = [540 + b for b in range(64)], [20 + b % 11 for b in range(64)]
    for b in (0, 5, 6, 40):
        lens[b] = b % 3
    check(lens, new, 512, 64, heads=1, group=2, dim=dim, form=form, dtype=F16)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_that_see_nothing_behind_many_splits(dim):
    """The same where a workgroup joins many partial results of a row."""
    check([35000, 0, 33000, 0], [1] * 4, 32768, 256, 2, 2, dim, INT8, F16)


@pytest.mark.parametrize("dim", [64, 128])
def test_scales_do_not_reach_rows_that_see_nothing(dim):
    batch, cache = shared_problem([600, 0, 590, 580], [1] * 4, 512, 64, enough_heads(4, 512, dim), dim, E4M3)
    cache.k_scale[int(batch.table[0, 2]), :, 1] = float("nan")
    Q = values(5, 4, cache.heads, dim, BF16)
    got = lg.gemv_kv_attend(Q, cache, *batch.tensors(False), shared=512)
    assert (got[1] == 0).all() and torch.isnan(got[[0, 2, 3]]).all()


@pytest.mark.parametrize("lens,new", [([601, 590, 570, 599], [1] * 4), ([0, 130, 100, 90], [1] * 4), ([17, 1, 0, 16], [1] * 4),
                                      ([601, 590, 570, 599, 33, 40, 500, 0], [3, 2, 5, 1, 9, 4, 1, 0]), ([70 - b for b in range(20)], [1] * 20)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_bytes_past_the_lengths(dim, lens, new):
    """Sequences that all end within the shared tokens: what lies behind the longest
    in its pages, NaN among it, does not matter."""
    shared, longest = 640, max(lens)
    batch, cache = shared_problem(lens, new, shared, 64, enough_heads(len(lens), shared, dim), dim, E4M3)
    batch.table[:] = batch.table[0]
    k, v = cache.k.view(torch.uint8), cache.v.view(torch.uint8)
    for at in range(longest, shared):
        page, i = int(batch.table[0, at // 64]), at % 64
        k[page, :, i] = 0xff if at % 2 else 0x7f
        v[page, :, i // 16, :, i % 16] = 0x7f if at % 3 else 0xff
        if at % 16 == 0:  # (blocks that nothing was written to)
            cache.k_scale[page, :, i // 16] = float("nan")
            cache.v_scale[page, :, i // 16] = float("inf")
    Q = values(3, batch.rows, cache.heads * 2, dim, F16)
    one_each = max(new) == 1
    assert taken_together(cache, cache.heads * 2, batch.rows, len(lens), batch.table.shape[1], one_each, 1 << 30)
    for window in (0, 50):
        got = lg.gemv_kv_attend(Q, cache, *batch.tensors(not one_each), window=window, shared=1 << 30)
        assert_close(got, *attend(f64(Q), PlainCache(cache), batch, dim ** -0.5, window, dtype=F16))


def test_padding_rows_stay():
    check([600, 590] * 4, [4, 3] * 4, 512, 64, padding=9)
    check([600, 590] * 4, [1, 1] * 4, 512, 64, padding=30)


def test_negative_and_zero_scale():
    check([600, 590, 570, 580], [1, 1, 1, 1], 512, 64, scale=-0.05)
    check([600, 590, 570, 580], [1, 1, 1, 1], 512, 64, scale=0.0)


@pytest.mark.parametrize("dim,group", [(64, 1), (64, 8), (128, 3), (256, 1)])
def test_the_largest_weight_of_single_tokens_is_whole(dim, group):
    """Where one shared token has the largest score and the only value, a single
    token's result is the formula's rounded once: its weight is 1 before the sum, not a
    number of fp16's 11 bits.  (Scores are whole multiples of a power of two but for the
    softmax scale's log2(e), 2^-24 of a score of 6 at most; the weight, the sum of some 4000
    others and the quotient round by 2^-24 a few hundred times.)"""
    shared, lens = 4096, [4100, 4200, 4130, 4097]
    heads = enough_heads(4, shared, dim)
    batch, cache = shared_problem(lens, [1] * 4, shared, 64, heads, dim, INT8)
    for t in (cache.k, cache.v):
        t.zero_()
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(1.0)
    value = torch.arange(dim, dtype=torch.int64) % 37 + 91
    for head in range(heads):  # (behind others that a wavefront weighs before it)
        at = 64 * (8 * (head % 8) + 4 + head % 4) + head % 64
        page, i = int(batch.table[0, at // 64]), at % 64
        cache.k[page, head, i, 0] = 1
        cache.v[page, head, i // 16, :, i % 16] = value.to(torch.int8).cuda()
    Q = torch.zeros(4, heads * group, dim, dtype=F16, device="cuda")
    Q[:, :, 0] = (torch.rand(4, heads * group, generator=torch.Generator().manual_seed(dim)) * 40 + 4).to(F16).cuda()
    assert taken_together(cache, heads * group, 4, 4, batch.table.shape[1], True, shared)
    got = f64(lg.gemv_kv_attend(Q, cache, *batch.tensors(False), scale=0.125, shared=shared))
    e = np.exp(f64(Q)[:, :, :1] * 0.125)
    want = value.numpy() * e / (e + np.array(lens)[:, None, None] - 1)
    half_step = 2.0 ** (np.floor(np.log2(want)) - 11)
    assert (np.abs(got - want) <= half_step + 2.0 ** -16 * want).all()


def test_too_little_to_share():
    """Where little is shared, or nothing, the call is the one without it."""
    for lens, new, shared in (([300, 290], [1, 1], 256), ([700], [1], 640), ([400, 330], [30, 7], 320), ([90] * 20, [1] * 20, 63)):
        batch, cache, Q, tensors = check(lens, new, shared, heads=2, group=4, together=False)
        assert torch.equal(lg.gemv_kv_attend(Q, cache, *tensors, shared=shared), lg.gemv_kv_attend(Q, cache, *tensors))


def test_missing_pages():
    """Shared tokens whose page is not there are not seen."""
    batch, cache = shared_problem([600, 590, 570, 599], [1] * 4, 512, 32, 64, 128, INT8)
    assert taken_together(cache, 64, 4, 4, batch.table.shape[1], True, 512)
    for bad in (-1, batch.pages, 1 << 30):
        batch.table[:, 3] = bad
        Q = values(1, 4, 64, 128, BF16)
        got = lg.gemv_kv_attend(Q, cache, *batch.tensors(False), shared=512)
        assert_close(got, *attend(f64(Q), PlainCache(cache), batch, 128 ** -0.5, dtype=BF16))


def test_more_rows_than_partial_results_are_kept_of():
    """Past 1 GiB of them the call is the one without shared tokens."""
    sequences, heads, group, dim, shared = 33000, 2, 8, 256, 512
    cache = filled(8 + sequences, heads, dim, 16, E4M3, 1)
    table = torch.empty(sequences, 33, dtype=torch.int32)
    table[:, :32] = torch.arange(32) % 8  # (pages may also be named twice)
    table[:, 32] = torch.arange(sequences) + 8
    table, lens = table.cuda(), (torch.arange(sequences, dtype=torch.int32) % 16 + 513).cuda()
    size = [lg.kv_attend_workspace_size(cache, heads * group, sequences, sequences, 33, shared=n) for n in (0, shared)]
    assert size[0] == size[1] and 8 * sequences * heads * group * dim > 1 << 30
    Q = torch.randn(sequences, heads * group, dim, device="cuda", dtype=BF16)
    assert torch.equal(lg.gemv_kv_attend(Q, cache, table, lens, shared=shared), lg.gemv_kv_attend(Q, cache, table, lens))


def test_more_shared_than_the_table_holds():
    batch, cache = shared_problem([512] * 4, [1] * 4, 512, 64, 64, 128, INT8)
    Q = values(1, 4, 64, 128, BF16)
    got = lg.gemv_kv_attend(Q, cache, *batch.tensors(False), shared=1 << 30)
    assert_close(got, *attend(f64(Q), PlainCache(cache), batch, 128 ** -0.5, dtype=BF16))


def test_hidden_blocks_that_are_not_finite():
    """A NaN scale reaches the rows that see its block, and no others."""
    batch, cache = shared_problem([800, 350, 790, 700], [1] * 4, 512, 64, 64, 128, E4M3)
    page = int(batch.table[0, 6])
    cache.k_scale[page, :, 1] = float("nan")        # tokens 400 to 415
    Q = values(2, 4, 64, 128, F16)
    got = lg.gemv_kv_attend(Q, cache, *batch.tensors(False), shared=512)
    assert torch.isnan(got[0]).all() and torch.isnan(got[2:]).all()
    want, bound = attend(f64(Q), PlainCache(cache), batch, 128 ** -0.5, dtype=F16)
    assert_close(got[1], want[1], bound[1])
    cache.k_scale[page, :, 1] = 1.0
    hidden = PlainCache(cache)  # (the window of 200 hides the block: its V scale has no part in the bound)
    cache.v_scale[page, :, 1] = float("inf")
    got = lg.gemv_kv_attend(Q, cache, *batch.tensors(False), shared=512, window=200)
    assert_close(got, *attend(f64(Q), hidden, batch, 128 ** -0.5, 200, 0, dtype=F16))


def test_a_row_does_not_depend_on_the_others():
    """A row's bits are the same whatever the other rows hold, and from call to
    call."""
    batch, cache, Q, tensors = check([700, 650, 660, 690], [1, 1, 1, 1], 640)
    first = lg.gemv_kv_attend(Q, cache, *tensors, shared=640)
    assert torch.equal(first, lg.gemv_kv_attend(Q, cache, *tensors, shared=640))
    other = Q.clone()
    other[1:] *= 30
    assert torch.equal(first[0], lg.gemv_kv_attend(other, cache, *tensors, shared=640)[0])
    other[1:] = float("nan")
    assert torch.equal(first[0], lg.gemv_kv_attend(other, cache, *tensors, shared=640)[0])


def test_workspace_and_graph():
    for lens, new in (([700, 650, 660, 690], [1] * 4), ([700, 650, 660, 690] * 2, [3, 1, 2, 1] * 2)):
        batch, cache, Q, tensors = check(lens, new, 640)
        one_each, heads = tensors[2] is None, cache.heads
        need = lg.kv_attend_workspace_size(cache, heads, batch.rows, len(lens), batch.table.shape[1], one_each=one_each, shared=640)
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
            Q.copy_(values(n, batch.rows, heads, 128, BF16))
            out.zero_()
            guard.fill_(255)  # (nothing of an earlier call's, NaN as numbers)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, lg.gemv_kv_attend(Q, cache, *tensors, shared=640)), n


def test_replayed_with_other_lengths():
    """A captured call whose sequences grow, end and leave their place empty."""
    for new in ([1] * 8, [3, 1, 2, 1, 1, 4, 1, 1]):
        batch, cache, Q, tensors = check([700, 650, 660, 690, 680, 645, 641, 700], new, 640, page_size=64)
        plain, lens = PlainCache(cache), tensors[1]
        out = torch.empty_like(Q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lg.gemv_kv_attend(Q, cache, *tensors, shared=640, out=out)
        for then in ([700, 0, 660, 690, 0, 645, 641, 1], [0] * 8, [2, 650, 0, 600, 640, 3, 64, 65], [690, 650, 660, 690, 680, 645, 641, 699]):
            lens.copy_(torch.tensor(then, dtype=torch.int32))
            batch.lens = then
            out.fill_(5.0)
            graph.replay()
            torch.cuda.synchronize()
            assert_close(out, *attend(f64(Q), plain, batch, 128 ** -0.5, dtype=BF16), str(then))
            assert torch.equal(out, lg.gemv_kv_attend(Q, cache, *tensors, shared=640)), then


def test_other_stream():
    batch, cache, Q, tensors = check([700, 650, 660, 690], [1, 1, 1, 1], 640)
    want = lg.gemv_kv_attend(Q, cache, *tensors, shared=640)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = lg.gemv_kv_attend(Q, cache, *tensors, shared=640, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_a_step_of_a_model():
    """A decode step and a prompt step as they are used: 4-bit products, norms and
    rotary positions, the append and the attention behind a shared prefix, against
    the same in 64 bits with the library's roundings between the operators."""
    from q4_helpers import product, rotary
    heads, group, dim, hidden, page, prefix = 8, 2, 64, 256, 16, 4100
    g = torch.Generator().manual_seed(3)
    width = (heads * group + 2 * heads) * dim
    W = torch.randint(0, 256, (width, hidden // 2), generator=g, dtype=torch.uint8).cuda()
    scale = (torch.rand(width, hidden // 32, generator=g) * 0.01).cuda()
    frequency, magnitude = lg.rotary_frequencies(dim, 10000.0, factor=2.0, original=2048)
    weight = [(1 + 0.1 * torch.randn(dim, generator=g)).cuda() for _ in range(2)]
    lens, new = [prefix + n for n in (30, 9, 20, 8, 30, 17, 1, 11)], [1] * 8
    for prompt in (False, True):
        if prompt:
            new = [20, 1, 9, 3, 30, 2, 1, 4]
        batch, cache = shared_problem(lens, new, prefix, page, heads, dim, INT8, seed=4)
        table, seq_lens, starts = batch.tensors(prompt)
        assert taken_together(cache, heads * group, batch.rows, 8, table.shape[1], not prompt, prefix)
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
