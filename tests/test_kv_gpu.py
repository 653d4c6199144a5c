"""The paged 8-bit key/value cache: the append and the attention over it,
against references in 64 bits (needs a GPU)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import memory_bound_gemv_f32_amd as lg
from fp8_helpers import Batch, PlainCache, assert_close, attend, decode

pytestmark = pytest.mark.gpu

INT8, E4M3 = torch.int8, torch.float8_e4m3fn
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def filled(pages, heads, dim, page_size, dtype, seed):
    """A cache of random bytes over the whole range (no NaN) and scales."""
    g = torch.Generator().manual_seed(seed)
    c = lg.KVCache.empty(pages, heads, dim, page_size=page_size, dtype=dtype)
    for t in (c.k, c.v):
        x = torch.randint(-127, 128, t.shape, generator=g, dtype=torch.int8)
        if dtype == E4M3:
            x = x.view(torch.uint8)
            x[(x & 127) == 127] = 3
        t.view(torch.uint8).copy_(x.view(torch.uint8))
    for t in (c.k_scale, c.v_scale):
        t.copy_(torch.exp2(torch.randint(-8, -4, t.shape, generator=g).float()) / (3 if dtype == E4M3 else 1))
    return c


def values(seed, rows, heads, dim, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, heads, dim, generator=g) * scale).to(dtype).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


def assert_same_cache(cache, plain, what=""):
    for name in ("k_scale", "v_scale", "k", "v"):
        t, want = getattr(cache, name), getattr(plain, name)
        got = f64(t) if name.endswith("scale") else decode(t)
        differ = ~((got == want) | (np.isnan(got) & np.isnan(want)))
        if differ.any():
            i = tuple(int(x) for x in np.argwhere(differ)[0])
            raise AssertionError(f"{what} {name}: {differ.sum()} differ, first {i}: got {got[i]!r} want {want[i]!r}")


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

APPENDS = [  # lengths after the call, new tokens
    ([1], [1]), ([16], [16]), ([17], [17]), ([40, 3, 16, 33], [1, 1, 1, 1]), ([5, 100, 64], [5, 37, 64]),
    ([20, 0, 31, 200], [4, 0, 16, 130]), ([15, 16, 17, 18], [15, 15, 15, 15]), ([300], [2])]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("form", [INT8, E4M3])
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append(case, form, dtype):
    lens, new = APPENDS[case]
    page_size, dim, heads = [16, 32, 64, 128, 256][case % 5], [64, 128, 256][case % 3], 1 + case % 3
    rng = np.random.default_rng(case)
    batch = Batch(lens, new, page_size, rng)
    cache = filled(batch.pages, heads, dim, page_size, form, case)
    plain = PlainCache(cache)
    K, V = values(1, batch.rows, heads, dim, dtype, 3.0), values(2, batch.rows, heads, dim, dtype, 0.05)
    one_each = all(m == 1 for m in new)
    lg.gemv_kv_append(cache, K, V, *batch.tensors(not one_each))
    plain.append(f64(K), f64(V), batch)
    assert_same_cache(cache, plain)


@pytest.mark.parametrize("form", [INT8, E4M3])
def test_append_token_by_token(form):
    """Growing scales round the earlier tokens again; the end state is the
    reference's, and in e4m3 that of one append of all tokens."""
    n, heads, dim, page = 37, 2, 64, 32
    K, V = values(3, n, heads, dim, F32), values(4, n, heads, dim, F32)
    up = torch.exp2(torch.arange(n, device="cuda") % 16 * 0.7)[:, None, None]
    K, V = K * up, V / up
    batch = Batch([n], [n], page, np.random.default_rng(0))
    cache = filled(batch.pages, heads, dim, page, form, 5)
    plain = PlainCache(cache)
    for t in range(n):
        step = Batch([t + 1], [1], page, np.random.default_rng(0))
        step.table = batch.table
        lg.gemv_kv_append(cache, K[t:t + 1], V[t:t + 1], *step.tensors(False))
        plain.append(f64(K[t:t + 1]), f64(V[t:t + 1]), step)
    assert_same_cache(cache, plain)


def test_append_edges():
    """Zeros, the smallest and largest magnitudes, values on the limit of a
    scale, infinities and NaN: the block's alone, until it starts anew."""
    heads, dim, page = 1, 64, 16
    for form, qmax in ((INT8, 127.0), (E4M3, 448.0)):
        for dtype in (F32, BF16):
            rows = []
            for top in (0.0, 1e-44, 1.1754944e-38, qmax, np.nextafter(np.float32(qmax), np.float32(1e9)), 2 * qmax,
                        1.0, 3.4e38):
                x = torch.zeros(16, heads, dim)
                x[3, 0, 5] = -float(top)
                x[4, 0, 6] = float(top) / 3
                rows.append(x)
            for bad in (float("inf"), float("-inf"), float("nan")):
                x = torch.ones(16, heads, dim)
                x[7, 0, 9] = bad
                rows.append(x)
            x = torch.cat(rows + [torch.ones(3, heads, dim)]).to(dtype).cuda()
            batch = Batch([len(x)], [len(x)], page, np.random.default_rng(1))
            cache = filled(batch.pages, heads, dim, page, form, 6)
            plain = PlainCache(cache)
            lg.gemv_kv_append(cache, x, x, *batch.tensors())
            plain.append(f64(x), f64(x), batch)
            assert_same_cache(cache, plain, (form, dtype))
            # a NaN in a block that has tokens already, then a good token, then the block anew
            for n, fill in ((len(x) + 1, float("nan")), (len(x) + 2, 1.0), (len(x) - 2, 2.0)):
                step = Batch([n], [1], page, np.random.default_rng(1))
                step.table = batch.table
                y = torch.full((1, heads, dim), fill, dtype=dtype, device="cuda")
                lg.gemv_kv_append(cache, y, y, *step.tensors())
                plain.append(f64(y), f64(y), step)
                assert_same_cache(cache, plain, (form, dtype, n))


def test_append_columns_of_a_wider_matrix_and_padding():
    heads, dim, page = 3, 128, 64
    batch = Batch([70, 12], [30, 12], page, np.random.default_rng(2))
    wide = values(7, batch.rows + 5, 2 * heads + 4, dim, F32)
    wide[batch.rows:] = float("nan")  # rows behind the last sequence are not read
    K, V = wide[:, 4:4 + heads], wide[:, 4 + heads:]
    cache = filled(batch.pages, heads, dim, page, E4M3, 8)
    plain = PlainCache(cache)
    lg.gemv_kv_append(cache, K, V, *batch.tensors())
    plain.append(f64(K[:batch.rows]), f64(V[:batch.rows]), batch)
    assert_same_cache(cache, plain)


def test_append_bad_pages_are_left_out():
    """Tokens of entries that are no page, or past the table, go nowhere."""
    heads, dim, page = 2, 64, 16
    batch = Batch([60, 40, 30], [60, 40, 5], page, np.random.default_rng(3))
    table, lens, starts = batch.tensors()
    cache = filled(batch.pages, heads, dim, page, INT8, 9)
    K, V = values(1, batch.rows, heads, dim, F32), values(2, batch.rows, heads, dim, F32)
    before = {n: getattr(cache, n).clone() for n in ("k", "v", "k_scale", "v_scale")}
    bad = torch.tensor([[-1, batch.pages, 2 ** 31 - 1, -2 ** 31]] * 3, dtype=torch.int32, device="cuda")
    lg.gemv_kv_append(cache, K, V, bad, lens, starts)
    lg.gemv_kv_append(cache, K, V, table[:, :0], lens, starts)
    # a length below the new tokens, negative or far too long: in bounds all the same
    for odd in ([2, 3, 1], [-5, 0, -2 ** 31], [2 ** 31 - 1] * 3):
        lg.gemv_kv_append(cache, K, V, bad, torch.tensor(odd, dtype=torch.int32, device="cuda"), starts)
    torch.cuda.synchronize()
    for n, t in before.items():
        assert torch.equal(getattr(cache, n).view(torch.uint8), t.view(torch.uint8)), n
    # of a sequence whose second page is bad the rest is written
    holes = batch.table.copy()
    holes[0, 1] = -7
    plain = PlainCache(cache)
    lg.gemv_kv_append(cache, K, V, torch.tensor(holes, device="cuda"), lens, starts)
    good = Batch([60, 40, 30], [60, 40, 5], page, np.random.default_rng(3))
    keep = {n: getattr(plain, n).copy() for n in ("k", "v", "k_scale", "v_scale")}
    plain.append(f64(K), f64(V), good)
    hole = batch.table[0, 1]
    for n, t in keep.items():
        getattr(plain, n)[hole] = t[hole]
    assert_same_cache(cache, plain)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def check_attend(batch, heads, group, dim, page, form, dtype, *, window=0, sinks=0, scale=None, seed=0, one_each=False,
                 cache=None, table=None):
    cache = filled(batch.pages, heads, dim, page, form, seed) if cache is None else cache
    Q = values(seed + 1, batch.rows, heads * group, dim, dtype)
    if table is not None:
        batch.table = table
    out = torch.full((batch.rows + 2, heads * group, dim), 9.0, dtype=dtype, device="cuda")
    lg.gemv_kv_attend(Q, cache, *batch.tensors(not one_each), window=window, sinks=sinks, scale=scale,
                      out=out[1:1 + batch.rows])
    want, bound = attend(f64(Q), PlainCache(cache), batch, dim ** -0.5 if scale is None else scale, window, sinks, dtype)
    assert (out[0] == 9.0).all() and (out[-1] == 9.0).all()
    assert_close(out[1:-1], want, bound, f"{batch.lens} {batch.new}")


DECODES = [([1], 1), ([15, 16, 17], 4), ([63, 64, 65, 1], 5), ([130, 0, 257], 8), ([1000], 16), ([2100, 7], 17),
           ([300, 301], 3)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("form", [INT8, E4M3])
@pytest.mark.parametrize("case", range(len(DECODES)))
def test_attend_single_tokens(case, form, dtype):
    lens, group = DECODES[case]
    page, dim, heads = [16, 32, 64, 128, 256][case % 5], [64, 128, 256][case % 3], 1 + case % 2
    batch = Batch(lens, [1] * len(lens), page, np.random.default_rng(case))
    check_attend(batch, heads, group, dim, page, form, dtype, one_each=True, seed=case)
    check_attend(batch, heads, group, dim, page, form, dtype, seed=case, window=20, sinks=3)


PROMPTS = [([5], [5], 1), ([20, 33], [20, 2], 4), ([130, 64, 90], [70, 64, 1], 2), ([200], [150], 3),
           ([40, 0, 70], [0, 0, 33], 5), ([300, 5], [17, 5], 8)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("form", [INT8, E4M3])
@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_attend_prompts(case, form, dtype):
    lens, new, group = PROMPTS[case]
    page, dim, heads = [16, 32, 64, 128, 256][case % 5], [128, 64, 128, 256][case % 4], 1 + case % 2
    batch = Batch(lens, new, page, np.random.default_rng(case))
    check_attend(batch, heads, group, dim, page, form, dtype, seed=case)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (17, 4), (64, 64), (65, 70), (100, 1), (1000, 5),
                                          (30, 1000)])
def test_attend_windows(window, sinks):
    batch = Batch([300, 90], [1, 1], 16, np.random.default_rng(1))
    check_attend(batch, 1, 4, 64, 16, E4M3, BF16, window=window, sinks=sinks, one_each=True)
    batch = Batch([300, 90], [140, 90], 16, np.random.default_rng(1))
    check_attend(batch, 1, 2, 64, 16, INT8, F16, window=window, sinks=sinks)


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.7])
def test_attend_scales(scale):
    batch = Batch([150], [40], 32, np.random.default_rng(1))
    check_attend(batch, 1, 2, 64, 32, E4M3, BF16, scale=scale)


def test_attend_long_context():
    batch = Batch([20011], [1], 128, np.random.default_rng(4))
    check_attend(batch, 1, 2, 128, 128, INT8, BF16, one_each=True)
    batch = Batch([9000, 3], [2, 2], 64, np.random.default_rng(4))
    check_attend(batch, 1, 3, 64, 64, E4M3, F16)


def test_attend_does_not_see_what_is_masked():
    """Bytes behind a sequence's end, unused pages, blocks whose scale is NaN
    or infinite and that a row does not see: none reaches a result."""
    heads, dim, page = 1, 64, 16
    for form in (INT8, E4M3):
        for dtype in (F16, BF16):
            batch = Batch([37, 70], [1, 33], page, np.random.default_rng(5))
            cache = filled(batch.pages, heads, dim, page, form, 5)
            Q = values(6, batch.rows, heads * 2, dim, dtype)
            args = (Q, cache, *batch.tensors())
            plain = lg.gemv_kv_attend(*args)
            # poison everything that no token of the batch holds
            last = int(batch.table[0, 2])
            cache.k.view(torch.uint8)[last, :, 5:] = 0x7F
            cache.v.view(torch.uint8)[last, :, :, :, 5:] = 0x7F
            used = set(batch.table[batch.table >= 0].tolist())
            for p in set(range(batch.pages)) - used:
                cache.k.view(torch.uint8)[p] = 0xFF
                cache.v.view(torch.uint8)[p] = 0xFF
                cache.k_scale[p] = float("nan")
                cache.v_scale[p] = float("inf")
            assert torch.equal(lg.gemv_kv_attend(*args), plain)
            # the last block of the second sequence: rows before it (positions 37 to 63) do not see it
            end = int(batch.table[1, 4])
            for name in ("k_scale", "v_scale"):
                for bad in (float("nan"), float("inf")):
                    keep = getattr(cache, name)[end].clone()
                    getattr(cache, name)[end] = bad
                    got = lg.gemv_kv_attend(*args)
                    assert torch.equal(got[:28], plain[:28]), (name, bad)
                    assert torch.isnan(got[28:]).all() or bad == float("inf"), (name, bad)
                    getattr(cache, name)[end] = keep


def test_attend_nan_query_is_its_rows_alone():
    batch = Batch([50], [20], 16, np.random.default_rng(6))
    cache = filled(batch.pages, 2, 64, 16, E4M3, 6)
    Q = values(7, 20, 4, 64, BF16)
    plain = lg.gemv_kv_attend(Q, cache, *batch.tensors())
    Q[3, 1] = float("nan")
    got = lg.gemv_kv_attend(Q, cache, *batch.tensors())
    assert torch.isnan(got[3, 1]).all()
    got[3, 1] = plain[3, 1]
    assert torch.equal(got, plain)


def test_attend_bad_pages():
    """Tokens in entries that are no page are not seen; a row that sees none is 0."""
    page, heads, dim = 16, 1, 64
    for new, one in (([1, 1], True), ([20, 3], False)):
        batch = Batch([100, 60], new, page, np.random.default_rng(7))
        table = batch.table.copy()
        table[0, 2], table[0, 6], table[1, :] = -5, batch.pages + 3, 2 ** 31 - 1
        check_attend(batch, heads, 4, dim, page, INT8, BF16, one_each=one, table=table)
    batch = Batch([100, 60], [1, 1], page, np.random.default_rng(7))
    cache = filled(batch.pages, heads, dim, page, INT8, 1)
    table, lens, _ = batch.tensors()
    Q = values(8, 2, 4, dim, F16)
    assert (lg.gemv_kv_attend(Q, cache, table[:, :0], lens) == 0).all()
    assert torch.equal(lg.gemv_kv_attend(Q, cache, table, lens + 0), lg.gemv_kv_attend(Q, cache, table, lens))
    # lengths that are negative or far past the table stay in bounds
    assert (lg.gemv_kv_attend(Q, cache, table, torch.tensor([-3, -2 ** 31], dtype=torch.int32, device="cuda")) == 0).all()
    lg.gemv_kv_attend(Q, cache, table, torch.full((2,), 2 ** 31 - 1, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()


def test_attend_padding_rows_are_left():
    batch = Batch([40, 30], [8, 5], 16, np.random.default_rng(8))
    cache = filled(batch.pages, 1, 64, 16, INT8, 8)
    Q = values(9, batch.rows + 6, 3, 64, BF16)
    Q[batch.rows:] = float("nan")
    out = torch.full_like(Q, 4.0)
    lg.gemv_kv_attend(Q, cache, *batch.tensors(), out=out)
    assert (out[batch.rows:] == 4.0).all()
    assert torch.equal(out[:batch.rows], lg.gemv_kv_attend(Q[:batch.rows], cache, *batch.tensors()))


def test_attend_strided_rows_and_shared_pages():
    """Q as columns of a wider matrix, out too; sequences that share pages."""
    batch = Batch([64, 64, 50], [1, 1, 1], 16, np.random.default_rng(9))
    batch.table[1] = batch.table[0]
    cache = filled(batch.pages, 2, 128, 16, E4M3, 9)
    wide = values(10, 3, 8 + 5, 128, F16)
    Q = wide[:, 3:11]
    Q[1] = Q[0]
    out = torch.zeros(3, 11, 128, dtype=F16, device="cuda")
    lg.gemv_kv_attend(Q, cache, *batch.tensors(False), out=out[:, 2:10])
    want, bound = attend(f64(Q), PlainCache(cache), batch, 128 ** -0.5, dtype=F16)
    assert_close(out[:, 2:10], want, bound)
    assert torch.equal(out[0], out[1]) and (out[:, :2] == 0).all() and (out[:, 10:] == 0).all()


def test_attend_repeats_and_workspace():
    batch = Batch([3000, 40], [1, 1], 64, np.random.default_rng(10))
    cache = filled(batch.pages, 2, 128, 64, INT8, 10)
    Q = values(11, 2, 8, 128, BF16)
    args = (Q, cache, *batch.tensors(False))
    plain = lg.gemv_kv_attend(*args)
    need = lg.kv_attend_workspace_size(cache, 8, 2, 2, batch.table.shape[1])
    assert need > 0
    ws = torch.full((need // 4 + 64,), float("nan"), device="cuda")
    ws[need // 4:] = 5.0
    for _ in range(3):
        assert torch.equal(lg.gemv_kv_attend(*args, workspace=ws[:need // 4]), plain)
    assert (ws[need // 4:] == 5.0).all()
    with pytest.raises(lg.GemvError):
        lg.gemv_kv_attend(*args, workspace=ws[:need // 4 - 1])


def test_attend_cache_past_4_gib():
    """Pages beyond 32-bit byte offsets."""
    heads, dim, page = 16, 256, 256
    pages = (1 << 32) // (heads * dim * page) + 40
    cache = lg.KVCache.empty(pages, heads, dim, page_size=page, dtype=INT8)
    batch = Batch([300], [1], page, np.random.default_rng(11))
    table = np.array([[pages - 1, pages - 5]], dtype=np.int32)
    small = filled(2, heads, dim, page, INT8, 12)
    for i in range(2):
        for n in ("k", "v", "k_scale", "v_scale"):
            getattr(cache, n)[int(table[0, i])] = getattr(small, n)[i]
    K, V = values(1, 1, heads, dim, BF16), values(2, 1, heads, dim, BF16)
    Q = values(3, 1, heads * 2, dim, BF16)
    outs = []
    for c, t in ((cache, table), (small, np.array([[0, 1]], dtype=np.int32))):
        batch.table = t
        lg.gemv_kv_append(c, K, V, *batch.tensors(False))
        outs.append(lg.gemv_kv_attend(Q, c, *batch.tensors(False)))
    assert torch.equal(outs[0], outs[1]) and torch.isfinite(outs[0]).all()
    for n in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(cache, n)[pages - 5], getattr(small, n)[1])


def test_refusals():
    c = filled(4, 2, 64, 16, INT8, 1)
    t = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    lens = torch.ones(3, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    K, Q = values(1, 3, 2, 64, F32), values(2, 3, 4, 64, F16)
    for args in ((K, K[:2], t, lens), (K[:, :1], K[:, :1], t, lens), (K, K.half(), t, lens),
                 (K, K, t.long(), lens), (K, K, t, lens.long()), (K, K, t, lens[:2]), (K, K, t, lens, starts[:3]),
                 (K[:2], K[:2], t, lens), (K, K, t.cpu(), lens), (K.transpose(0, 1), K.transpose(0, 1), t, lens),
                 (K[..., :32], K[..., :32], t, lens)):
        with pytest.raises(ValueError):
            lg.gemv_kv_append(c, *args)
    with pytest.raises(TypeError):
        lg.gemv_kv_append(c, K.double(), K.double(), t, lens)
    with pytest.raises(TypeError):
        lg.gemv_kv_attend(Q.float(), c, t, lens)
    for kw in (dict(out=torch.empty_like(Q.bfloat16())), dict(out=torch.empty_like(Q)[:2])):
        with pytest.raises(ValueError):
            lg.gemv_kv_attend(Q, c, t, lens, **kw)
    for kw in (dict(window=-1), dict(sinks=-1), dict(scale=float("nan"))):
        with pytest.raises(lg.GemvError):
            lg.gemv_kv_attend(Q, c, t, lens, **kw)
    with pytest.raises(lg.GemvError):
        lg.gemv_kv_attend(Q[:, :3], c, t, lens)
    with pytest.raises(ValueError):
        lg.KVCache.empty(4, 2, 64, page_size=48)
    with pytest.raises(ValueError):
        lg.KVCache(c.k, c.v, c.k_scale[:2], c.v_scale)
    with pytest.raises(TypeError):
        lg.KVCache(c.k, c.v.view(torch.uint8), c.k_scale, c.v_scale)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

class Layer:
    """The attention half of a decode step on 8-bit weights and an 8-bit cache."""

    def __init__(self, form, hidden=512, q_heads=8, heads=2, dim=64, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.q_heads, self.heads, self.dim, self.form = q_heads, heads, dim, form
        width = (q_heads + 2 * heads) * dim
        self.wqkv = lg.gemv_fp8_quantise((torch.randn(width, hidden, generator=g) * 0.05).cuda(), 128)
        self.wo = lg.gemv_fp8_quantise((torch.randn(hidden, q_heads * dim, generator=g) * 0.05).cuda(), 128)

    def __call__(self, x, cache, table, lens, starts=None):
        qkv = lg.gemv_fp8(*self.wqkv, *lg.gemv_fp8_quantise(x), out_dtype=BF16)
        qkv = qkv.view(len(x), -1, self.dim)
        q, k, v = qkv.split((self.q_heads, self.heads, self.heads), dim=1)
        lg.gemv_kv_append(cache, k, v, table, lens, starts)
        o = lg.gemv_kv_attend(q, cache, table, lens, starts)
        return lg.gemv_fp8(*self.wo, *lg.gemv_fp8_quantise(o.view(len(x), -1)))


@pytest.mark.parametrize("form", [INT8, E4M3])
def test_a_layer_in_prompts_and_single_tokens(form):
    """A prompt at once, then single tokens, in a batch of two; each call's
    attention against the reference on the cache as it then is."""
    layer = Layer(form)
    cache = lg.KVCache.empty(12, 2, 64, page_size=32, dtype=form)
    cache.k.view(torch.uint8).fill_(0x7F)  # a new cache's contents do not matter
    cache.v.view(torch.uint8).fill_(0x7F)
    cache.k_scale.fill_(float("nan"))
    cache.v_scale.fill_(float("nan"))
    table = torch.tensor([[3, 7, 1], [0, 5, 9]], dtype=torch.int32, device="cuda")
    lens, new = [21, 40], [21, 40]
    g = torch.Generator().manual_seed(3)
    for step in range(5):
        batch = Batch(lens, new, 32, np.random.default_rng(0))
        batch.table = table.cpu().numpy()
        x = torch.randn(sum(new), 512, generator=g).to(BF16).cuda()
        args = (table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                torch.tensor(batch.starts, device="cuda") if step == 0 else None)
        y = layer(x, cache, *args)
        qkv = lg.gemv_fp8(*layer.wqkv, *lg.gemv_fp8_quantise(x), out_dtype=BF16).view(len(x), -1, 64)
        o = lg.gemv_kv_attend(qkv[:, :8], cache, *args)
        want, bound = attend(f64(qkv[:, :8]), PlainCache(cache), batch, 64 ** -0.5)
        assert_close(o, want, bound)
        assert torch.equal(y, lg.gemv_fp8(*layer.wo, *lg.gemv_fp8_quantise(o.reshape(len(x), -1))))
        assert torch.isfinite(y).all()
        lens, new = [n + 1 for n in lens], [1, 1]


def test_a_captured_step_replays():
    """One decode step in a graph, replayed over growing sequences with the
    program's own work between: every replay equals the eager step."""
    layer = Layer(E4M3, seed=4)
    caches = [lg.KVCache.empty(70, 2, 64, page_size=16, dtype=E4M3) for _ in range(2)]
    for c in caches:  # whole scale tensors are compared, blocks that no step writes among them
        c.k_scale.zero_()
        c.v_scale.zero_()
    table = torch.randperm(70, device="cuda")[:66].view(2, 33).to(torch.int32)
    prompt = torch.randn(305, 512, generator=torch.Generator().manual_seed(4)).to(BF16).cuda()
    x = torch.zeros(2, 512, dtype=BF16, device="cuda")
    lens = torch.tensor([300, 5], dtype=torch.int32, device="cuda")
    for c in caches:
        layer(prompt, c, table, lens, torch.tensor([0, 300, 305], dtype=torch.int32, device="cuda"))
    lens += 1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x, caches[0], table, lens)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(x, caches[0], table, lens)
    g = torch.Generator().manual_seed(5)
    for step in range(40):
        x.copy_(torch.randn(2, 512, generator=g).to(BF16))
        lens.copy_(torch.tensor([301 + step, 6 + step], dtype=torch.int32))
        graph.replay()
        want = layer(x, caches[1], table, lens)
        if step % 3 == 0:
            torch.cuda.synchronize()
        assert torch.isfinite(want).all() and torch.equal(y, want), step
        for n in ("k_scale", "v_scale"):
            torch.testing.assert_close(getattr(caches[0], n), getattr(caches[1], n), rtol=0, atol=0, equal_nan=True)


def test_calls_on_other_streams():
    layer = Layer(INT8, seed=6)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    lens = torch.tensor([50, 64], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 50, 114], dtype=torch.int32, device="cuda")
    x = torch.randn(114, 512, device="cuda").to(BF16)
    caches = [lg.KVCache.empty(8, 2, 64, page_size=16) for _ in range(4)]
    want = layer(x, caches[0], table, lens, starts)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s, c in zip(streams, caches[1:]):
        with torch.cuda.stream(s):
            got.append(layer(x, c, table, lens, starts))
    torch.cuda.synchronize()
    for y in got:
        assert torch.equal(y, want)


def test_call_on_a_given_stream_takes_its_memory_there():
    """With ``stream`` the result and the workspace come from that stream's
    memory, so that what else has had them, or has them next, is in order."""
    side = torch.cuda.Stream()
    cache = filled(64, 2, 64, 256, INT8, 3)
    table = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([64 * 256], dtype=torch.int32, device="cuda")
    q = values(1, 1, 8, 64, BF16)
    need = lg.kv_attend_workspace_size(cache, 8, 1, 1, 64)
    assert need > 0
    want = lg.gemv_kv_attend(q, cache, table, lens)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got = lg.gemv_kv_attend(q, cache, table, lens, stream=side)
    x = torch.randn(2, 256, device="cuda")
    torch.cuda.synchronize()
    held = lg.gemv_fp8_quantise(x, stream=side)
    weight = lg.gemv_fp8_quantise(x, 128, stream=side)
    y = lg.gemv_fp8(*weight, *held, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert torch.equal(y, lg.gemv_fp8(*weight, *held))
    own = [s for s in torch.cuda.memory_snapshot() if s["stream"] == side.cuda_stream]
    for t in (got, *held, *weight, y):
        assert any(s["address"] <= t.data_ptr() < s["address"] + s["total_size"] for s in own)
    assert sum(s["total_size"] for s in own) >= need


def test_attend_lengths_and_sinks_up_to_an_int():
    """Positions up to 2^31 - 2 (one page that the whole table repeats), and
    sinks that cover everything."""
    cache = filled(1, 2, 64, 256, INT8, 4)
    q = values(2, 1, 4, 64, F16)
    top = 2**31 - 1
    wide = torch.zeros(1, 2**31 // 256, dtype=torch.int32, device="cuda")
    lens = torch.tensor([top], dtype=torch.int32, device="cuda")
    here = torch.tensor([top % 256], dtype=torch.int32, device="cuda")
    # the same tokens at positions 155 .. 254 of the page
    got = lg.gemv_kv_attend(q, cache, wide, lens, window=100)
    want = lg.gemv_kv_attend(q, cache, wide[:, :1].contiguous(), here, window=100)
    assert torch.equal(got, want)
    table = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    lens[0] = 1000
    want = lg.gemv_kv_attend(q, cache, table, lens)
    for sinks in (1000, top - 64, top):
        got = lg.gemv_kv_attend(q, cache, table, lens, window=70, sinks=sinks)
        # (the same chunks in the same order)
        assert torch.equal(got, want), sinks
    for kw in (dict(window=2**31), dict(sinks=2**32 + 5), dict(window=5 - 2**32)):
        with pytest.raises(ValueError):
            lg.gemv_kv_attend(q, cache, table, lens, **kw)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (600, 20)])
def test_attend_prompts_split_over_tokens(dim, window, sinks):
    """Wavefronts with rows of their own whose tokens several workgroups share;
    a short sequence beside a long one."""
    batch = Batch([1500, 3, 790], [45, 3, 60], 64, np.random.default_rng(dim))
    cache = filled(batch.pages, 1, dim, 64, INT8, 1)
    table = batch.tensors()[0]
    assert lg.kv_attend_workspace_size(cache, 2, batch.rows, 3, table.shape[1], one_each=False, window=window,
                                       sinks=sinks) > 0
    for form, dtype in ((INT8, F16), (E4M3, BF16)):
        check_attend(batch, 1, 2, dim, 64, form, dtype, window=window, sinks=sinks, seed=dim)
