"""Norms and rotary positions of query and key heads against a reference in 64
bits (needs a GPU)."""

from __future__ import annotations

from fractions import Fraction

import numpy as np
import pytest
import torch

import memory_bound_gemv_f32_amd as lg
from q4_helpers import assert_close, rotary

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(lens, new, q_heads, heads, dim, dtype, pairs, norm, seed=0, pad=0, padding=0):
    """Queries and keys as columns of one matrix, with ``padding`` rows behind
    the last sequence's."""
    g = torch.Generator().manual_seed(seed)
    rows = sum(new) + padding
    both = torch.randn(rows, (q_heads + 2 * heads) * dim + pad, generator=g).to(dtype).cuda()
    Q = both[:, :q_heads * dim].unflatten(1, (q_heads, dim))
    K = both[:, q_heads * dim:(q_heads + heads) * dim].unflatten(1, (heads, dim))
    frequency = torch.exp(-torch.arange(pairs).double() * (np.log(10000.0) / max(pairs, 1))).float().cuda()
    weights = [(1 + 0.3 * torch.randn(dim, generator=g)).cuda() if norm else None for _ in range(2)]
    starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    positions = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)] or [[]])
    return Q, K, frequency, weights, torch.tensor(lens, dtype=torch.int32, device="cuda"), starts, positions


def check(lens, new, q_heads, heads, dim, dtype, pairs, norm=False, interleaved=False, magnitude=1.0, q_dtype=None,
          k_dtype=None, with_starts=True, eps=1e-6, **kw):
    Q, K, frequency, (wq, wk), seq_lens, starts, positions = make(lens, new, q_heads, heads, dim, dtype, pairs, norm, **kw)
    before = Q.clone(), K.clone()
    q, k = lg.gemv_rotary(Q, K, frequency, seq_lens, starts if with_starts else None, q_weight=wq, k_weight=wk, eps=eps,
                          magnitude=magnitude, interleaved=interleaved, q_dtype=q_dtype, k_dtype=k_dtype)
    assert torch.equal(Q, before[0]) and torch.equal(K, before[1])
    n = len(positions)
    for x, w, y, out in ((Q, wq, q, q_dtype or dtype), (K, wk, k, k_dtype or dtype)):
        assert y.dtype == out and y.shape == x.shape
        assert_close(y[:n], *rotary(x[:n], positions, frequency, w, eps, magnitude, interleaved, out),
                     f"{lens} {dim} {pairs} {dtype} {out} {norm} {interleaved}")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
def test_sizes(dtype, interleaved):
    """Head sizes of every mapping, part or all of them rotated."""
    for n, (dim, pairs) in enumerate([(2, 1), (2, 0), (6, 2), (8, 4), (40, 8), (64, 32), (64, 16), (66, 33), (80, 40), (96, 12),
                                      (128, 64), (128, 32), (128, 31), (130, 64), (192, 96), (256, 128), (256, 32),
                                      (258, 100), (384, 192), (512, 256), (510, 255), (512, 0)]):
        check([40, 3, 17], [5, 3, 1], (n % 5) + 1, (n % 3) + 1, dim, dtype, pairs, norm=n % 2 == 0,
              interleaved=interleaved, seed=n, pad=n % 3)


@pytest.mark.parametrize("dtype,q_dtype,k_dtype", [(F32, F16, F32), (F32, BF16, BF16), (F32, F32, F16), (F16, F16, F32),
                                                   (BF16, F32, BF16), (BF16, F16, F16)])
def test_types(dtype, q_dtype, k_dtype):
    check([100, 7], [1, 1], 32, 8, 128, dtype, 64, norm=True, q_dtype=q_dtype, k_dtype=k_dtype, with_starts=False)
    check([100, 7], [60, 7], 5, 1, 96, dtype, 20, q_dtype=q_dtype, k_dtype=k_dtype, interleaved=True, magnitude=1.3)


def test_far_positions():
    """Positions up to an int's end keep the angle's fraction (against 64-bit
    mantissas), a rounding of 64 bits' turns would not."""
    for lens in ([131071, 1 << 20], [1 << 24, (1 << 24) + 1], [(1 << 31) - 1, (1 << 30) + 12345]):
        check(lens, [3, 2], 4, 2, 64, F32, 32)


PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798214808651")


def test_large_frequencies():
    """Frequencies far above 1, and positions up to an int's end: the angle keeps fp32's
    bits of its place in the turn (against whole numbers, with 100 digits of pi)."""
    pairs = 24
    frequency = torch.tensor([1.7 ** (3 * i) * (1 + 0.01 * i) for i in range(pairs)])  # to 2^52
    for length in (3, 1000, (1 << 20) + 7, (1 << 31) - 1):
        x = torch.zeros(2, 1, 2 * pairs)
        x[:, :, :pairs] = 1.0
        y, _ = lg.gemv_rotary(x.cuda(), None, frequency.cuda(), torch.tensor([length], dtype=torch.int32, device="cuda"),
                              torch.tensor([0, 2], dtype=torch.int32, device="cuda"))
        for row in range(2):
            for i in range(pairs):
                turns = (length - 2 + row) * Fraction(float(frequency[i])) / (2 * PI)
                place = 2 * np.pi * float(turns - round(turns))
                # the angle's place rounded to fp32, a sine or cosine within two steps, two products and a sum
                bound = (np.pi + 2 + 3) * 2.0 ** -24
                got = [float(y[row, 0, i]), float(y[row, 0, i + pairs])]
                assert abs(got[0] - np.cos(place)) <= bound and abs(got[1] - np.sin(place)) <= bound, (length, row, i)


def test_batches():
    """Empty sequences, one or thousands of them, more tokens than wavefronts at work."""
    check([5, 0, 0, 9, 0], [2, 0, 0, 4, 0], 3, 1, 64, BF16, 32)
    check([0, 0, 4], [0, 0, 4], 3, 1, 64, BF16, 32)
    check([1], [1], 1, 1, 64, BF16, 32, with_starts=False)
    lens = list(range(1, 301))
    check(lens, [1] * 300, 2, 1, 64, F16, 16, with_starts=False, norm=True)
    check(lens, [1 + n % 3 if n >= 3 else 1 for n in range(1, 301)], 2, 2, 64, F16, 16, norm=True)
    check([3000, 5000], [3000, 1000], 8, 2, 128, BF16, 64, norm=True)


@pytest.mark.parametrize("dim,pairs", [(128, 64), (100, 30)])
def test_in_place_and_padding(dim, pairs):
    """In place, with rows behind the last sequence's left as they were."""
    Q, K, frequency, (wq, wk), lens, starts, positions = make([9, 30], [4, 7], 6, 2, dim, BF16, pairs, True, padding=5)
    want = lg.gemv_rotary(Q, K, frequency, lens, starts, q_weight=wq, k_weight=wk)
    q0, k0 = Q.clone(), K.clone()
    q, k = lg.gemv_rotary(Q, K, frequency, lens, starts, q_weight=wq, k_weight=wk, q_out=Q, k_out=K)
    assert q.data_ptr() == Q.data_ptr()
    assert torch.equal(Q[:11], want[0][:11]) and torch.equal(K[:11], want[1][:11])
    assert torch.equal(Q[11:], q0[11:]) and torch.equal(K[11:], k0[11:])


def test_queries_alone_and_one_weight():
    Q, K, frequency, (wq, wk), lens, starts, positions = make([9], [9], 6, 2, 128, F16, 64, True)
    both = lg.gemv_rotary(Q, K, frequency, lens, starts, q_weight=wq)
    q, none = lg.gemv_rotary(Q, None, frequency, lens, starts, q_weight=wq)
    assert none is None and torch.equal(q, both[0])
    assert_close(both[1], *rotary(K, positions, frequency, None, 1e-6, 1.0, False, F16))


def test_norm_edges():
    """Heads of zeros, tiny and large values, infinities and NaN: each its own."""
    dim = 128
    x = torch.randn(6, 2, dim)
    x[0] = 0
    x[1] *= 1e-12
    x[2] *= 1e12
    x[3, 0, 5], x[4, 1, 77] = float("inf"), float("nan")
    x = x.cuda()
    lens = torch.tensor([6], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    w = torch.ones(dim, device="cuda")
    frequency, _ = lg.rotary_frequencies(dim)
    y, _ = lg.gemv_rotary(x, None, frequency, lens, starts, q_weight=w, eps=1e-6)
    bad = torch.zeros(6, 2, dtype=torch.bool, device="cuda")
    bad[3, 0] = bad[4, 1] = True
    keep = ~bad
    want, bound = rotary(x, np.arange(6), frequency, w, 1e-6, 1.0, False, F32)
    got = y.double().cpu().numpy()
    assert (np.abs(got - want) <= bound)[keep.cpu().numpy()].all()
    assert torch.isnan(y[3, 0]).any() and torch.isnan(y[4, 1]).all()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,pairs", [(128, 32), (64, 8), (100, 30), (66, 0), (258, 100)])
def test_values_that_are_not_rotated_stay(dim, pairs, interleaved, dtype):
    """Behind the rotated ones every value is the input's own, whatever it and
    its neighbours are: infinities, NaN, zeros of both signs."""
    at = 2 * pairs
    x = torch.randn(5, 3, dim, generator=torch.Generator().manual_seed(dim))
    odd = torch.tensor([float("inf"), 0.0, 1.5, float("nan"), -0.0, -1.0, -float("inf"), -0.0, 0.0, -2.0])
    for row in range(5):
        for i, v in enumerate(odd.roll(row)):
            x[row, :, at + (3 * i + row) % (dim - at)] = v
    x = x.to(dtype).cuda()
    lens = torch.tensor([9], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    frequency = torch.rand(pairs, generator=torch.Generator().manual_seed(1)).cuda()
    y, k = lg.gemv_rotary(x, x, frequency, lens, starts, interleaved=interleaved, magnitude=1.25, k_dtype=F32)
    for out, same in ((y, x), (k, x.float())):
        nan = torch.isnan(same[:, :, at:])
        assert torch.equal(torch.isnan(out[:, :, at:]), nan)
        kind = torch.int32 if out.dtype == F32 else torch.int16
        bits = [t[:, :, at:].contiguous().view(kind)[~nan] for t in (out, same)]
        assert torch.equal(*bits)
    if pairs:
        want, bound = rotary(x[:, :, :at], np.arange(4, 9), frequency, None, 1e-6, 1.25, interleaved, dtype)
        assert_close(y[:, :, :at], want, bound)


def test_frequencies():
    f, m = lg.rotary_frequencies(64, 10000.0)
    assert m == 1.0 and torch.equal(f.cpu(), (10000.0 ** (-torch.arange(32).double() / 32)).float())
    g, m = lg.rotary_frequencies(64, 10000.0, factor=4.0)
    assert m == 1.0 and torch.equal(g.cpu(), (10000.0 ** (-torch.arange(32).double() / 32) / 4).float())
    h, m = lg.rotary_frequencies(64, 10000.0, factor=4.0, original=4096)
    assert abs(m - (1 + 0.1 * np.log(4))) < 1e-12
    turns = 4096 * f.double().cpu().numpy() / (2 * np.pi)
    ratio = (h.double() / f.double()).cpu().numpy()
    assert np.allclose(ratio[turns > 64], 1, atol=1e-6) and np.allclose(ratio[turns < 0.5], 0.25, atol=1e-6)
    assert (np.diff(ratio) <= 1e-6).all() and len(f) == 32


def test_streams_and_graphs():
    Q, K, frequency, (wq, wk), lens, starts, _ = make([9, 30], [4, 7], 6, 2, 128, BF16, 64, True)
    want = lg.gemv_rotary(Q, K, frequency, lens, starts, q_weight=wq)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = lg.gemv_rotary(Q, K, frequency, lens, starts, q_weight=wq, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = torch.empty_like(want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lg.gemv_rotary(Q, None, frequency, lens, starts, q_weight=wq, q_out=out)
    for n in range(3):
        lens += 17
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, lg.gemv_rotary(Q, None, frequency, lens, starts, q_weight=wq)[0]), n


def test_helper_refusals():
    Q, K, frequency, (wq, wk), lens, starts, _ = make([9, 30], [4, 7], 6, 2, 128, BF16, 64, True)
    call = lg.gemv_rotary
    for bad in (lambda: call(Q, K[:5], frequency, lens, starts), lambda: call(Q, K.float(), frequency, lens, starts),
                lambda: call(Q, K[:, :, :64], frequency, lens, starts), lambda: call(Q, K, frequency.double(), lens, starts),
                lambda: call(Q, K, frequency, lens), lambda: call(Q, K, frequency, lens.long(), starts),
                lambda: call(Q, K, frequency, lens, starts[:2]), lambda: call(Q, K, frequency, lens, starts, q_weight=wq[:5]),
                lambda: call(Q, None, frequency, lens, starts, k_weight=wk), lambda: call(Q, K, frequency.cpu(), lens, starts),
                lambda: call(Q, K, frequency, lens, starts, q_out=K),
                lambda: call(Q, K, frequency, lens, starts, q_out=Q, q_dtype=F32)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        call(Q.double(), K.double(), frequency, lens, starts)
    with pytest.raises(lg.GemvError):
        call(Q, K, torch.ones(65, device="cuda"), lens, starts)
    with pytest.raises(lg.GemvError):
        call(Q, K, frequency, lens, starts, eps=-1.0)
