"""The attention over the paged 8-bit cache at the ends of its range, against
the reference in 64 bits (needs a GPU)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import memory_bound_gemv_f32_amd as lg
from fp8_helpers import EPS, Batch, PlainCache, assert_close
from test_kv_gpu import BF16, E4M3, F16, INT8, check_attend, f64, filled, values

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


def attend_terms(Q, plain, batch, scale, dtype):
    """(O, bound) in 64 bits, the bound in the row's own terms.

    Scores are off by d and weights by a factor within exp(2d), as for
    fp8_helpers.attend, and a term (a weight times its block's V scale) is
    rounded to fp16's 11 bits, half a step being 2^-11 of it, unless it is below
    2^-20 of the row's largest: then to half of fp16's smallest step in the
    row's unit, 2^-25 times at most 2^-6 of the largest (or 2^-126, the least
    unit).  A term meets the token's byte; the rest is fp32 (a few steps for each
    weight, the sum's n, the unit's changes) and the result's own rounding."""
    out, bound = np.zeros(Q.shape), np.zeros(Q.shape)
    rows, q_heads, dim = Q.shape
    heads = plain.k.shape[1]
    group, half = q_heads // heads, EPS[dtype] / 2
    for b, (n, m) in enumerate(zip(batch.lens, batch.new)):
        for h in range(heads):
            at = [(int(batch.table[b, p // batch.page_size]), p % batch.page_size // 16, min(16, n - p)) for p in range(0, n, 16)]
            k = np.concatenate([plain.block("k", p, h, s)[:c] * plain.k_scale[p, h, s] for p, s, c in at])
            byte = np.concatenate([plain.block("v", p, h, s)[:c] for p, s, c in at])
            vs = np.concatenate([np.full(c, plain.v_scale[p, h, s]) for p, s, c in at])
            for i in range(m):
                see = n - m + i + 1
                for g in range(h * group, (h + 1) * group):
                    q = Q[int(batch.starts[b]) + i, g]
                    s = scale * (k[:see] @ q)
                    d = (dim + 8) * 2.0 ** -23 * scale * (np.abs(k[:see]) @ np.abs(q)).max()
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    t = w * vs[:see]
                    o, spread = t @ byte[:see], t @ np.abs(byte[:see])
                    low = (2.0 ** -31 * t.max() + 2.0 ** -151 * w.max()) * np.abs(byte[:see]).sum(0)
                    rel = 2.0 ** -11 + 2 * d + (see + 64) * 2.0 ** -23
                    row = int(batch.starts[b]) + i
                    out[row, g] = o
                    bound[row, g] = 1.01 * (rel * spread + low) + half * np.abs(o) + (2.0 ** -25 if dtype == F16 else 1e-37)
    return out, bound


def check_terms(cache, batch, Q, one_each):
    dim = Q.shape[2]
    got = lg.gemv_kv_attend(Q, cache, *batch.tensors(not one_each))
    want, bound = attend_terms(f64(Q), PlainCache(cache), batch, dim ** -0.5, Q.dtype)
    assert_close(got, want, bound, f"{batch.lens} {batch.new}")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,new,group", [([1000, 90], [1, 1], 4), ([9000], [1], 2), ([300, 70], [12, 3], 2), ([400, 40], [60, 40], 2)])
@pytest.mark.parametrize("up", [12, 20, 26, 60])
def test_large_value_scales_of_little_weight(up, lens, new, group, dim):
    """Blocks whose V scale is 2^up times the others' and whose weights are next
    to nothing: what has the weight keeps its bits."""
    form, dtype = ((INT8, BF16), (E4M3, F16))[up // 4 % 2]
    batch = Batch(lens, new, 16, np.random.default_rng(up))
    cache = filled(batch.pages, 1, dim, 16, form, up)
    Q = values(up, batch.rows, group, dim, dtype).abs()
    step = 2.0 ** -(up + 8) if dtype == F16 else 1.0  # (the results are within fp16)
    cache.v_scale.mul_(step)
    for b in range(len(lens)):
        pages = torch.tensor(batch.table[b][batch.table[b] >= 0].astype(np.int64), device="cuda")
        for j, far in ((0, 30.0), (len(pages) // 2, 50.0)):
            # every score of the block is -far, give or take a part of it
            cache.k.view(torch.uint8)[pages[j]] = 0xC0 if form == INT8 else 0xB8  # int8 -64, e4m3 -1.0
            cache.k_scale[pages[j]] = far / (64 if form == INT8 else 1) / (0.8 * dim ** 0.5)
            cache.v_scale[pages[j]] *= 2.0 ** up
    check_terms(cache, batch, Q, all(m == 1 for m in new))


@pytest.mark.parametrize("lens,new,group", [([500, 200], [1, 1], 4), ([9000], [1], 2), ([300, 70], [12, 3], 2), ([400, 40], [60, 40], 2)])
@pytest.mark.parametrize("form", [INT8, E4M3])
def test_value_scales_over_many_powers(form, lens, new, group):
    """V scales over 2^40, in every order along a row, some of them zero."""
    for dim in (64, 128, 256):
        batch = Batch(lens, new, 16, np.random.default_rng(dim))
        cache = filled(batch.pages, 1, dim, 16, form, dim)
        g = torch.Generator().manual_seed(dim)
        cache.v_scale.copy_(torch.exp2(torch.randint(-30, 11, cache.v_scale.shape, generator=g).float()))
        cache.v_scale[torch.rand(cache.v_scale.shape, generator=g).cuda() < 0.1] = 0.0
        cache.k_scale.mul_(4.0)
        check_terms(cache, batch, values(dim, batch.rows, group, dim, BF16), all(m == 1 for m in new))


@pytest.mark.parametrize("lens,new", [([600, 90], [1, 1]), ([9000], [1]), ([300, 70], [60, 2])])
def test_a_long_tail_of_small_weights_counts(lens, new):
    """One token of each 64 has nearly all the weight and no value; the others,
    each 2^-26.4 of it, make the result."""
    dim = 64
    batch = Batch(lens, new, 64, np.random.default_rng(1))
    for form in (INT8, E4M3):
        cache = filled(batch.pages, 1, dim, 64, form, 1)
        one = 1 if form == INT8 else 0x38
        cache.k.view(torch.uint8).fill_(0)
        cache.v.view(torch.uint8).fill_(one)
        cache.k_scale.fill_(26.4 * np.log(2.0) * dim ** 0.5)
        cache.v_scale.fill_(1024.0)
        cache.k.view(torch.uint8)[:, 0, 0, 0] = one
        cache.v.view(torch.uint8)[:, 0, 0, :, 0] = 0
        for dtype in (F16, BF16):
            Q = torch.ones(batch.rows, 2, dim, dtype=dtype, device="cuda")
            check_terms(cache, batch, Q, all(m == 1 for m in new))


def test_results_near_the_largest_number():
    """Values near fp32's largest, of which the result is the mean and not the sum."""
    for form, byte in ((INT8, 127), (E4M3, 0x7E)):
        for lens, new in (([300, 40], [1, 1]), ([9000], [1]), ([300, 40], [60, 2])):
            batch = Batch(lens, new, 16, np.random.default_rng(2))
            cache = filled(batch.pages, 1, 64, 16, form, 2)
            cache.v.view(torch.uint8).fill_(byte)
            cache.v_scale.fill_(2.0 ** (120 if form == INT8 else 118))
            check_terms(cache, batch, values(3, batch.rows, 2, 64, BF16), all(m == 1 for m in new))
