"""Products with 4-bit weights and group scales against a reference in 64 bits
(needs a GPU)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import memory_bound_gemv_f32_amd as lg
from q4_helpers import assert_close, f64, product
from q4_variants import CASES, FAR

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def problem(M, K, nvec, group, dtype, zero=True, bias=False, seed=0, pad=0, shift=0):
    """Random codes, scales, zeros and vectors; pad: elements between rows; shift:
    elements in front of the first (so that no row is aligned)."""
    g = torch.Generator().manual_seed(seed * 1000003 + M * 31 + K * 7 + nvec)
    groups = -(-K // group)

    def within(t):
        wide = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype)
        wide[:, :t.shape[1]] = t
        flat = torch.cat((torch.zeros(shift, dtype=t.dtype), wide.flatten())).cuda()
        return flat[shift:].view(wide.shape)[:, :t.shape[1]]
    Q = within(torch.randint(0, 256, (M, -(-K // 2)), generator=g, dtype=torch.uint8))
    scale = within((torch.rand(M, groups, generator=g) * 0.02 + 0.001).to(dtype))
    z = within(torch.randint(0, 16, (M, groups), generator=g, dtype=torch.uint8)) if zero else None
    X = within(torch.randn(nvec, K, generator=g).to(dtype))
    b = torch.randn(M, generator=g).cuda() if bias else None
    return Q, scale, X, b, z


def check(M, K, nvec, group, dtype, out_dtype=F32, what="", **kw):
    Q, scale, X, b, z = problem(M, K, nvec, group, dtype, **kw)
    y = lg.gemv_q4(Q, scale, X, b, zero=z, group=group, out_dtype=out_dtype)
    assert y.dtype == out_dtype and y.shape == (nvec, M)
    assert_close(y, *product(Q, scale, X, b, z, group, out_dtype), f"{M}x{K} {nvec} {group} {dtype} {out_dtype} {kw} {what}")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_sizes(dtype, group):
    """Rows, columns and vectors on both sides of every tile."""
    for n, (M, K, nvec) in enumerate([(1, 1, 1), (1, 2, 1), (3, 31, 2), (16, 32, 1), (17, 33, 15), (5, 64, 16),
                                      (40, 127, 17), (64, 128, 1), (33, 129, 5), (100, 255, 33), (16, 256, 64),
                                      (50, 1000, 3), (129, 2049, 1), (70, 4096, 20)]):
        check(M, K, nvec, group, dtype, out_dtype=(F32, dtype)[n % 2], zero=n % 3 != 0, bias=n % 2 == 1, seed=n)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_many_vectors(dtype):
    for n, (M, K, nvec) in enumerate([(256, 512, 65), (200, 384, 128), (130, 640, 129), (300, 1031, 200), (128, 4096, 256),
                                      (1000, 256, 500)]):
        check(M, K, nvec, (32, 64, 128)[n % 3], dtype, out_dtype=(dtype, F32)[n % 2], zero=n % 2 == 0, bias=n % 2 == 0, seed=n)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_very_many_vectors(dtype, group):
    """Tiles of 256 rows, of 64, 112 and 128 vectors, the last ones not full; the
    same rows and vectors where they are not aligned, or the last columns no chunk."""
    for n, (M, K, nvec, kw) in enumerate([(2100, 256, 1100, {}), (4090, 384, 1101, {}), (8000, 128, 1000, {}),
                                          (2100, 256, 1100, dict(pad=1, shift=3)), (2100, 300, 1100, {}),
                                          (2100, 256, 1100, dict(pad=16, shift=16))]):
        check(M, K, nvec, group, dtype, out_dtype=(dtype, F32)[n % 2], zero=n % 2 == 0, bias=n % 3 == 0, seed=n, **kw)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_every_kernel(case, group):
    """Every kernel that the rule names, of every type and group, at ragged sizes."""
    dtype, family, M, K, nvec, pad, shift = CASES[case]
    Q, scale, X, b, z = problem(M, K, nvec, group, dtype, zero=case % 3 != 0, bias=case % 2 == 0, seed=case,
                                pad=0 if pad >= FAR else pad, shift=shift)
    if pad >= FAR:
        wide = torch.zeros(nvec, pad, dtype=dtype, device="cuda")
        wide[:, :K] = X
        X = wide[:, :K]
    out_dtype = (F32, F16, BF16)[(case + group // 32) % 3]
    y = lg.gemv_q4(Q, scale, X, b, zero=z, group=group, out_dtype=out_dtype)
    assert_close(y, *product(Q, scale, X, b, z, group, out_dtype), f"{CASES[case]} {group}")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_layouts(dtype):
    """Rows apart and unaligned, outputs that are columns of a wider matrix."""
    for n, (M, K, nvec) in enumerate([(20, 300, 1), (33, 256, 4), (70, 1000, 18), (200, 520, 150)]):
        for pad, shift in ((1, 0), (3, 1), (16, 5)):
            check(M, K, nvec, (32, 128)[n % 2], dtype, pad=pad, shift=shift, seed=n, bias=True)
    Q, scale, X, b, z = problem(50, 200, 9, 64, dtype)
    wide = torch.full((9, 70), 7.0, device="cuda", dtype=BF16)
    y = lg.gemv_q4(Q, scale, X, b, wide[:, 11:61], zero=z, group=64)
    assert y.data_ptr() == wide[:, 11:61].data_ptr()
    assert_close(wide[:, 11:61], *product(Q, scale, X, b, z, 64, BF16))
    assert (wide[:, :11] == 7).all() and (wide[:, 61:] == 7).all()


def test_single_vector_form():
    Q, scale, X, b, z = problem(100, 512, 1, 128, F16, bias=True)
    y = lg.gemv_q4(Q, scale, X[0], b, zero=z)
    assert y.shape == (100,) and y.dtype == F32
    assert torch.equal(y, lg.gemv_q4(Q, scale, X, b, zero=z)[0])
    out = torch.empty(100, device="cuda", dtype=F16)
    assert lg.gemv_q4(Q, scale, X[0], b, out, zero=z) is out
    assert_close(out[None], *product(Q, scale, X, b, z, 128, F16))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_whole_numbers_are_exact(dtype):
    """Small whole numbers in every place: each product and sum is exact in
    fp32, so the result is exact, whatever the layout and mapping."""
    g = torch.Generator().manual_seed(5)
    for M, K, nvec in ((48, 200, 1), (33, 1024, 16), (64, 333, 40), (160, 640, 130)):
        for group in (32, 64, 128):
            groups = -(-K // group)
            Q = torch.randint(0, 256, (M, -(-K // 2)), generator=g, dtype=torch.uint8).cuda()
            scale = torch.exp2(torch.randint(-2, 3, (M, groups), generator=g).float()).to(dtype).cuda()
            z = torch.randint(0, 256, (M, groups), generator=g, dtype=torch.uint8).cuda()
            X = torch.randint(-3, 4, (nvec, K), generator=g).to(dtype).cuda()
            for zero in (None, z):
                y = lg.gemv_q4(Q, scale, X, zero=zero, group=group)
                want, _ = product(Q, scale, X, None, zero, group, F32)
                assert np.array_equal(f64(y), want), (M, K, nvec, group, zero is None)


def test_fp32_parts():
    """fp32 vectors keep all their bits: values with 24 of them against one
    weight, at every magnitude down to where the parts leave the normal range."""
    K = 128
    Q = torch.full((16, K // 2), 0x88, dtype=torch.uint8, device="cuda")
    Q[:, 0] = 0x89  # column 0 is 1, all others 0
    scale = torch.ones(16, 1, device="cuda")
    bits = torch.arange(1, 100, dtype=torch.int32) * 0x00151413 % 0x800000
    for exponent in (24, 100, 127, 200, 254):
        x = (bits + (exponent << 23)).view(torch.float32)
        X = torch.zeros(len(x), K)
        X[:, 0] = torch.where(torch.arange(len(x)) % 2 == 0, x, -x)
        y = lg.gemv_q4(Q, scale, X.cuda())
        assert torch.equal(y.cpu(), X[:, :1].expand(-1, 16)), exponent


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_not_finite(dtype):
    """An infinity or NaN in a vector, or in a scale, reaches its own results
    and no others."""
    for nvec in (3, 40, 150):
        M, K = 40, 320
        Q, scale, X, b, z = problem(M, K, nvec, 32, dtype, seed=nvec)
        Q[:, 35] = 0x99
        z[:, 2] = 3
        X[1, 70], X[2, 70] = float("inf"), float("nan")
        scale[7, 3], scale[9, 4] = float("inf"), float("nan")
        y = f64(lg.gemv_q4(Q, scale, X, zero=z, group=32))
        want, bound = product(Q, scale, X, None, z, 32, F32)
        plain = np.ones(y.shape, dtype=bool)
        plain[1:3] = plain[:, 7] = plain[:, 9] = False
        assert (np.abs(y - want) <= bound)[plain].all()
        ordinary = [m for m in range(M) if m not in (7, 9)]
        assert np.isposinf(y[1, ordinary]).all() and np.isnan(y[2]).all() and np.isnan(y[:, 9]).all()
        assert not np.isfinite(y[:, 7]).any()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_large_tiles_at_their_edges(dtype, group):
    """Very many vectors: whole numbers are exact with every zero; what is not finite
    reaches its own results; the same bits on every call and when captured."""
    M, K, nvec = 2100, 256, 1100
    groups = K // group
    g = torch.Generator().manual_seed(group)
    Q = torch.randint(0, 256, (M, K // 2), generator=g, dtype=torch.uint8).cuda()
    scale = torch.exp2(torch.randint(-2, 3, (M, groups), generator=g).float()).to(dtype).cuda()
    z = torch.randint(0, 256, (M, groups), generator=g, dtype=torch.uint8).cuda()
    X = torch.randint(-3, 4, (nvec, K), generator=g).to(dtype).cuda()
    for zero in (None, z):
        y = lg.gemv_q4(Q, scale, X, zero=zero, group=group)
        assert np.array_equal(f64(y), product(Q, scale, X, None, zero, group, F32)[0]), zero is None
    wide = torch.full((nvec, M + 20), 7.0, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lg.gemv_q4(Q, scale, X, None, wide[:, 9:M + 9], zero=z, group=group)
    for n in range(3):
        X.copy_(torch.randint(-3, 4, (nvec, K), generator=g).to(dtype))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(wide[:, 9:M + 9], lg.gemv_q4(Q, scale, X, zero=z, group=group)), n
    assert (wide[:, :9] == 7).all() and (wide[:, M + 9:] == 7).all()
    Q[:, 35] = 0x99  # columns 70 and 71
    z[:, 70 // group] = 3
    X[1, 70], X[1098, 70] = float("inf"), float("nan")
    scale[7, -1], scale[2099, 0] = float("inf"), float("nan")
    y = f64(lg.gemv_q4(Q, scale, X, zero=z, group=group))
    want = product(Q, scale, X, None, z, group, F32)[0]
    plain = np.ones(y.shape, dtype=bool)
    plain[1] = plain[1098] = plain[:, 7] = plain[:, 2099] = False
    assert (y == want)[plain].all()
    ordinary = [m for m in range(M) if m not in (7, 2099)]
    assert np.isposinf(y[1, ordinary]).all() and np.isnan(y[1098]).all() and np.isnan(y[:, 2099]).all()
    assert not np.isfinite(y[np.abs(want[:, 7]) != 0, 7]).any()


def test_nan_with_low_bits_only():
    X = torch.zeros(1, 32)
    X.view(torch.int32)[0, 4] = 0x7f800001
    Q = torch.full((16, 16), 0x99, dtype=torch.uint8, device="cuda")
    assert torch.isnan(lg.gemv_q4(Q, torch.ones(16, 1, device="cuda"), X.cuda(), group=32)).all()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("M,K,nvec", [((1 << 20) + 77, 40, 2), (33, 70, (1 << 15) + 45), ((1 << 20) + 5, 9, 1)])
def test_more_than_one_launch_holds(M, K, nvec, dtype):
    """Rows past 2^20 and vectors past 2^15 go to launches of their own."""
    for n, (zero, bias) in enumerate([(True, True), (False, False)]):
        check(M, K, nvec, 32, dtype, out_dtype=(F32, dtype)[n], zero=zero, bias=bias, seed=n)


@pytest.mark.parametrize("dtype,group", [(BF16, 128), (F16, 32), (F32, 64)])
@pytest.mark.parametrize("K", [2 ** 31 - 1, 2 ** 31 - 128])
def test_rows_up_to_an_int(K, dtype, group):
    """The longest rows: all zero but for whole numbers at the start, the middle and the
    end, so the result is exact."""
    g = torch.Generator().manual_seed(K % 1000 + group)
    M, groups = 2, -(-K // group)
    Q = torch.zeros(M, -(-K // 2), dtype=torch.uint8, device="cuda")
    scale = torch.ones(M, groups, dtype=dtype, device="cuda")
    X = torch.zeros(1, K, dtype=dtype, device="cuda")
    want = np.zeros((1, M))
    for at in (0, 2 ** 30 - 50, (K - 201) // 2 * 2):
        n = min(300, K - at)
        codes = torch.randint(0, 256, (M, -(-n // 2)), generator=g, dtype=torch.uint8)
        Q[:, at // 2:at // 2 + codes.shape[1]] = codes.cuda()
        for part in range(at // group, min((at + n - 1) // group + 1, groups)):
            scale[:, part] = 2.0 ** (part % 3)
        x = torch.randint(-3, 4, (n,), generator=g)
        X[0, at:at + n] = x.to(dtype).cuda()
        q = f64(codes).astype(int)
        w = np.stack((q & 15, q >> 4), 2).reshape(M, -1)[:, :n] - 8
        want += ((w * 2.0 ** (((at + np.arange(n)) // group) % 3)) @ f64(x))[None]
    assert np.array_equal(f64(lg.gemv_q4(Q, scale, X, group=group)), want)


def test_empty():
    for M, K, nvec in ((0, 64, 3), (5, 64, 0), (5, 0, 3)):
        Q = torch.empty(M, K // 2, dtype=torch.uint8, device="cuda")
        scale, X = torch.empty(M, K // 32, dtype=F16, device="cuda"), torch.empty(nvec, K, dtype=F16, device="cuda")
        b = torch.randn(M, device="cuda")
        y = lg.gemv_q4(Q, scale, X, b, group=32)
        assert y.shape == (nvec, M)
        assert torch.equal(y, b.expand(nvec, M))
        if K == 0:
            assert (lg.gemv_q4(Q, scale, X, group=32) == 0).all()


def test_bytes_past_the_rows_are_not_used():
    """What lies between rows, in the last byte's upper half and behind the last
    row's end does not matter."""
    M, K = 20, 77
    Q, scale, X, b, z = problem(M, K, 3, 32, BF16, pad=9)
    y = lg.gemv_q4(Q, scale, X, zero=z, group=32)
    Q2 = Q.clone()
    Q2[:, 38] |= 0xf0
    assert torch.equal(y, lg.gemv_q4(Q2, scale, X, zero=z, group=32))


def test_streams_and_graphs():
    Q, scale, X, b, z = problem(300, 1024, 4, 128, BF16, bias=True)
    want = lg.gemv_q4(Q, scale, X, b, zero=z, out_dtype=BF16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = lg.gemv_q4(Q, scale, X, b, zero=z, out_dtype=BF16, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lg.gemv_q4(Q, scale, X, b, out, zero=z)
    for n in range(3):
        X.copy_(torch.randn(X.shape, device="cuda"))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, lg.gemv_q4(Q, scale, X, b, zero=z, out_dtype=BF16)), n


def test_helper_refusals():
    Q, scale, X, b, z = problem(8, 64, 2, 32, F16)
    for bad in (lambda: lg.gemv_q4(Q, scale, X, group=48), lambda: lg.gemv_q4(Q, scale, X, group=64),
                lambda: lg.gemv_q4(Q[:, :31], scale, X, group=32), lambda: lg.gemv_q4(Q, scale.float(), X, group=32),
                lambda: lg.gemv_q4(Q, scale, X, zero=z[:, :1], group=32),
                lambda: lg.gemv_q4(Q, scale, X, zero=z.to(torch.int8), group=32),
                lambda: lg.gemv_q4(Q, scale, X, out=torch.empty(2, 9, device="cuda"), group=32),
                lambda: lg.gemv_q4(Q, scale, X, torch.zeros(7, device="cuda"), group=32),
                lambda: lg.gemv_q4(Q.cpu(), scale, X, group=32)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lg.gemv_q4(Q.to(torch.int8), scale, X, group=32),
                lambda: lg.gemv_q4(Q, scale, X.double(), group=32),
                lambda: lg.gemv_q4(Q, scale, X, out_dtype=torch.float64, group=32)):
        with pytest.raises(TypeError):
            bad()
