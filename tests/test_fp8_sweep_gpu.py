"""A seeded sweep of the 8-bit operators over sizes, layouts and batches
against the references in 64 bits (needs a GPU): odd sizes and pitches, empty
sequences, padding rows, tables that are too short or hold entries that are no
page, windows and first tokens of any size."""

from __future__ import annotations

import math
import random

import numpy as np
import pytest
import torch

import memory_bound_gemv_f32_amd as lg
from fp8_helpers import Batch, PlainCache, assert_close, attend, product, product_bound
from test_fp8_gpu import operand
from test_kv_gpu import BF16, E4M3, F16, F32, INT8, assert_same_cache, f64, filled, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("seed", range(8))
def test_attend(seed):
    r = random.Random(seed)
    for n in range(25):
        count, one = r.choice((1, 2, 3, 7, 70)), r.random() < 0.5
        most = 3000 if count < 4 else 700 if count < 10 else 120
        lens = [r.choice((0, 1, r.randint(1, most))) for _ in range(count)]
        new = [1] * count if one else [r.choice((0, 1, min(k, r.randint(0, 60)))) for k in lens]
        heads, group, dim = r.choice((1, 2, 3)), r.choice((1, 2, 4, 8, 17, 33)), r.choice((64, 128, 256))
        window, sinks = r.choice((0, 0, 1, r.randint(1, most))), r.choice((0, 1, 4, r.randint(0, most), 10 ** 6))
        batch = Batch(lens, new, r.choice((16, 32, 64, 128, 256)), np.random.default_rng(n), width=r.choice((0, 3)))
        if r.random() < 0.3:
            batch.table = batch.table[:, :r.randint(1, batch.table.shape[1])].copy()
        if r.random() < 0.3:
            batch.table[r.randrange(count), r.randrange(batch.table.shape[1])] = r.choice((-1, batch.pages, 2 ** 31 - 1))
        form, dtype = r.choice((INT8, E4M3)), r.choice((F16, BF16))
        rows = batch.rows + (0 if one else r.choice((0, 3)))
        cache = filled(batch.pages, heads, dim, batch.page_size, form, n)
        Q = values(n, rows, heads * group + 2, dim, dtype)[:, 1:-1]
        wide = torch.full((rows, heads * group + 3, dim), 7.0, dtype=dtype, device="cuda")
        out = wide[:, 2:-1]
        lg.gemv_kv_attend(Q, cache, *batch.tensors(not one), window=window, sinks=sinks, out=out)
        want, bound = attend(f64(Q[:batch.rows]), PlainCache(cache), batch, dim ** -0.5, window, sinks, dtype)
        # (fp16's smallest step, of which a small result's rounding is half)
        bound = bound + (2.0 ** -25 if dtype == F16 else 0.0)
        what = (seed, n, lens, new, heads, group, dim, batch.page_size, window, sinks, form, dtype, one)
        assert (wide[:, :2] == 7.0).all() and (wide[:, -1] == 7.0).all() and (out[batch.rows:] == 7.0).all(), what
        assert_close(out[:batch.rows], want, bound, what)


@pytest.mark.parametrize("seed", range(4))
def test_append(seed):
    r = random.Random(seed)
    for n in range(15):
        count, one = r.choice((1, 2, 5, 100)), r.random() < 0.4
        new = [1] * count if one else [r.choice((0, 1, r.randint(0, 70))) for _ in range(count)]
        lens = [m + r.choice((0, 0, r.randint(0, 90))) for m in new]
        heads, dim, form = r.choice((1, 3)), r.choice((64, 128, 256)), r.choice((INT8, E4M3))
        batch = Batch(lens, new, r.choice((16, 32, 256)), np.random.default_rng(n))
        dtype = r.choice((F32, F16, BF16))
        cache = filled(batch.pages, heads, dim, batch.page_size, form, n)
        plain = PlainCache(cache)
        K = values(1, batch.rows, 2 * heads, dim, dtype, 3.0)[:, heads:]
        V = values(2, batch.rows, heads, dim, dtype, 0.05)
        lg.gemv_kv_append(cache, K, V, *batch.tensors(not one))
        plain.append(f64(K), f64(V), batch)
        assert_same_cache(cache, plain, (seed, n))


@pytest.mark.parametrize("seed", range(6))
def test_product(seed):
    r = random.Random(seed)
    def spread(low, high):
        return int(math.exp(r.uniform(math.log(low), math.log(high + 1))))
    for n in range(20):
        tokens, M, K = spread(1, 1200), spread(1, 6000), spread(1, 5000)
        if tokens * M * K > 2e9:
            tokens = 1 + tokens % 40
        K = K if r.random() < 0.5 else -(-K // 16) * 16
        off, out = r.choice((0, 0, 1, 16)), r.choice((F32, F16, BF16))
        W, ws = operand(n, M, K + off, 128)
        X, xs = operand(n + 1, tokens, K + off, 1)
        blocks = -(-K // 128)
        W, X, ws, xs = W[:, off:], X[:, off:], ws[:, :blocks], xs[:, :blocks]
        bias = values(n, 1, 1, M, F32)[0, 0] if r.random() < 0.5 else None
        wide = torch.full((tokens + 2, M + 3), 5.0, dtype=out, device="cuda")
        lg.gemv_fp8(W, ws, X, xs, bias, out=wide[1:-1, 1:1 + M])
        want, size = product(W, ws, X, xs, bias)
        what = (seed, n, tokens, M, K, off, out)
        if out != F16 or np.abs(want).max() < 60000:
            assert_close(wide[1:-1, 1:1 + M], want, product_bound(size, want, K, out), what)
        rest = wide.cpu()
        rest[1:-1, 1:1 + M] = 5.0
        assert (rest == 5.0).all(), what
