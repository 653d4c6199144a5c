"""The attention over the paged 8-bit cache at the ends of its range, against
the reference in 64 bits (needs a GPU)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import memory_bound_gemv_f32_amd as lg
from fp8_helpers import Batch
from test_kv_gpu import BF16, E4M3, F16, INT8, check_attend, filled, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("new", [1, 3, 70])
@pytest.mark.parametrize("window,sinks", [(16, 4), (500, 40), (16, 4000), (300, 10 ** 6), (2000, 130), (0, 0)])
def test_sequences_longer_than_their_table(window, sinks, new):
    """Tokens past a sequence's row of the table are not there: under a window
    with first tokens that stay visible too, in calls that are split over their
    tokens and in calls that are not."""
    for width, lens in ((16, [10000, 700, 1030]), (32, [2500, 2049, 90]), (1, [200, 64, 33])):
        batch = Batch(lens, [min(new, n) for n in lens], 64, np.random.default_rng(width))
        for form, dtype in ((INT8, BF16), (E4M3, F16)):
            check_attend(batch, 2, 4, 128, 64, form, dtype, window=window, sinks=sinks, one_each=new == 1,
                         table=batch.table[:, :width].copy())


@pytest.mark.parametrize("window,sinks", [(0, 0), (16, 4), (16, 2 ** 31 - 1)])
def test_a_table_of_no_pages(window, sinks):
    cache = filled(4, 2, 128, 64, INT8, 1)
    table = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    for lens in ([100, 5], [2 ** 31 - 1, 1]):
        lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for starts, rows in ((None, 2), (torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda"), 4)):
            out = torch.full((rows, 8, 128), 9.0, dtype=F16, device="cuda")
            lg.gemv_kv_attend(values(1, rows, 8, 128, F16), cache, table, lens, starts, window=window, sinks=sinks, out=out)
            assert (out == 0).all()


@pytest.mark.parametrize("one_each", [True, False])
@pytest.mark.parametrize("form", [INT8, E4M3])
def test_value_scales_of_any_size(form, one_each):
    """A caller's own scales, down to the smallest subnormal fp32 and zero: a
    block of tiny values in front, alone or behind ordinary ones."""
    for tiny in (0.0, 2.0 ** -149, 2.0 ** -140, 2.0 ** -128, 2.0 ** -127, 2.0 ** -126):
        for where in (slice(0, 1), slice(0, None), slice(3, None)):
            batch = Batch([150, 64], [1, 1] if one_each else [40, 3], 16, np.random.default_rng(3))
            cache = filled(batch.pages, 1, 64, 16, form, 3)
            for b in range(2):
                pages = torch.tensor(batch.table[b][batch.table[b] >= 0][where].astype(np.int64), device="cuda")
                cache.v_scale[pages] = tiny
            check_attend(batch, 1, 4, 64, 16, form, BF16, one_each=one_each, cache=cache)


@pytest.mark.parametrize("new,group", [([30, 1, 1, 1], 1), ([30, 2], 2), ([60, 3], 2)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_later_tokens_do_not_change_a_rows_bits(dim, new, group):
    """Of a row that does not see a block not even the rounding depends on it:
    not where the rows next to it do, in the same step, and find a far larger
    score or value scale there."""
    batch = Batch([9 * 64, 70, 70, 70][:len(new)], new, 16, np.random.default_rng(5))
    for form, dtype in ((INT8, BF16), (E4M3, F16)):
        cache = filled(batch.pages, 1, dim, 16, form, 5)
        cache.k_scale.mul_(0.25)
        Q = values(6, batch.rows, group, dim, dtype)
        args = (Q, cache, *batch.tensors())
        plain = lg.gemv_kv_attend(*args)
        last = int(batch.table[0, 9 * 4 - 1])  # positions 560 to 575, of which rows from new - 16 on see some
        for name, by in (("k_scale", 64.0), ("v_scale", 64.0), ("v_scale", 2.0 ** 21)):
            keep = getattr(cache, name)[last].clone()
            getattr(cache, name)[last] *= by
            got = lg.gemv_kv_attend(*args)
            getattr(cache, name)[last] = keep
            assert not torch.equal(got[new[0] - 16:new[0]], plain[new[0] - 16:new[0]])
            assert torch.equal(got[:new[0] - 16], plain[:new[0] - 16]), (name, by)
            assert torch.equal(got[new[0]:], plain[new[0]:]), (name, by)
