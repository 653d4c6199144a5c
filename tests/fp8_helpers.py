"""References in 64 bits for the 8-bit operators, on the host: e4m3 decoding,
the block quantiser's formula, the block-scaled product, a dictionary of what
a paged cache holds, and attention over it.  They share no code with the
library."""

from __future__ import annotations

import numpy as np
import torch

EPS = {torch.float32: 2.0 ** -23, torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7}
QMAX = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


def e4m3_values() -> np.ndarray:
    """The values of the bytes 0 to 255, from the format's definition."""
    out = []
    for byte in range(256):
        e, m = byte >> 3 & 15, byte & 7
        x = np.nan if (byte & 127) == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out.append(-x if byte & 128 else x)
    return np.array(out)


GRID = e4m3_values()


def decode(t: torch.Tensor) -> np.ndarray:
    """A tensor of int8 or e4m3 as float64."""
    t = t.detach().cpu().contiguous()
    if t.dtype == torch.int8:
        return t.numpy().astype(np.float64)
    return GRID[t.view(torch.uint8).numpy()]


def round8(x: np.ndarray, dtype) -> np.ndarray:
    """float64 values rounded to the nearest that the format holds (ties to even)."""
    x = np.clip(x, -QMAX[dtype], QMAX[dtype])
    if dtype == torch.int8:
        return np.rint(x)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -40))), -6) - 3)
    return np.clip(np.rint(x / step) * step, -448, 448)


def quantise(x: torch.Tensor, block_rows: int):
    """The quantiser's formula in IEEE fp32, block by block: (values as
    float64, scales float32)."""
    x = x.detach().cpu().float().numpy()
    rows, K = x.shape
    q = np.zeros((rows, K))
    scale = np.zeros((-(-rows // block_rows), -(-K // 128)), dtype=np.float32)
    for i in range(scale.shape[0]):
        for j in range(scale.shape[1]):
            at = (slice(i * block_rows, (i + 1) * block_rows), slice(j * 128, (j + 1) * 128))
            s = np.maximum(np.abs(x[at]).max() / np.float32(448), np.float32(2.0 ** -126))
            scale[i, j] = s
            q[at] = round8((x[at] * (np.float32(1) / s)).astype(np.float64), torch.float8_e4m3fn)
    return q, scale


def product(W, w_scale, X, x_scale, bias=None):
    """(Y, Σ|terms|) in 64 bits of the block-scaled product of torch tensors."""
    def full(q, s, rows):
        s = s.detach().cpu().double().numpy().repeat(rows, 0)[:q.shape[0]].repeat(128, 1)[:, :q.shape[1]]
        return decode(q) * s
    w, x = full(W, w_scale, 128), full(X, x_scale, 1)
    y, size = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        b = bias.detach().cpu().double().numpy()
        y, size = y + b, size + np.abs(b)
    return y, size


def product_bound(size, y, K, dtype):
    """A block's 128 exact products are added in fp32 (at most 128 roundings;
    one step each where an adder truncates), its sum scaled (two roundings) and
    added to the other blocks' (K/128, and 16 wavefronts'), the bias once, and
    the result rounded to its type by half a step.  For fp16 and bf16 results of
    more than 32 tokens the matrix cores align each 8 e4m3 products to the
    largest of them and cut what lies below 2^-13 of it: each of the other 7
    loses at most 2^-13 of the largest, which is at most the 8's Σ|products|."""
    chain = 2 * 128 + K / 128 + 16 + 4
    fine = chain * 2.0 ** -24 * size
    if dtype != torch.float32 and y.shape[0] > 32:
        fine = fine + 7 * 2.0 ** -13 * size
    half = EPS[dtype] / 2 if dtype != torch.float32 else 0.0
    tiny = 2.0 ** -25 if dtype == torch.float16 else 1e-37
    return fine * (1 + half) + half * np.abs(y) + tiny


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------

class Batch:
    """Shuffled pages of random sequences, on the host."""

    def __init__(self, lens, new, page_size, rng, spare=3, width=0):
        self.lens, self.new, self.page_size = list(lens), list(new), page_size
        need = [-(-n // page_size) for n in lens]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        self.table = np.full((len(lens), max([width, 1] + need)), -1, dtype=np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.rows = int(self.starts[-1])

    def tensors(self, with_starts=True):
        dev = "cuda"
        return (torch.tensor(self.table, device=dev), torch.tensor(self.lens, dtype=torch.int32, device=dev),
                torch.tensor(self.starts, device=dev) if with_starts else None)


class PlainCache:
    """A cache in 64 bits on the host: values over scale and scales, in the
    library's layout."""

    def __init__(self, cache):
        self.dtype = cache.k.dtype
        self.page_size = cache.page_size
        self.k, self.v = decode(cache.k), decode(cache.v)
        self.k_scale = cache.k_scale.cpu().double().numpy()
        self.v_scale = cache.v_scale.cpu().double().numpy()

    def block(self, which, page, head, sub):
        """(16, dim) view of a block's values."""
        if which == "k":
            return self.k[page, head, sub * 16:(sub + 1) * 16]
        return self.v[page, head, sub].T

    def append(self, K, V, batch: Batch):
        """K, V: float64 (rows, heads, dim)."""
        for which, x, scales in (("k", K, self.k_scale), ("v", V, self.v_scale)):
            for b, (n, m) in enumerate(zip(batch.lens, batch.new)):
                pos = n - m
                row = int(batch.starts[b])
                while pos < n:
                    page = int(batch.table[b, pos // self.page_size])
                    sub, off = pos % self.page_size // 16, pos % 16
                    take = min(16 - off, n - pos)
                    for h in range(x.shape[1]):
                        new = x[row:row + take, h]
                        blk = self.block(which, page, h, sub)
                        if not np.isfinite(new).all() or (off and np.isnan(scales[page, h, sub])):
                            blk[:off + take] = 0.0
                            scales[page, h, sub] = np.nan
                            continue
                        need = 2.0 ** -126
                        while np.abs(new).max() > need * QMAX[self.dtype]:
                            need *= 2
                        old = scales[page, h, sub]
                        s = max(need, old) if off else need
                        # the formula's ratio, reciprocal and products are IEEE fp32; for the
                        # powers of two that the append chooses they are exact, for a
                        # caller's own scales they round (3·fl(1/6) is 1/2 in fp32, a tie)
                        f = np.float32
                        blk[:off] = round8((blk[:off].astype(f) * (f(old) / f(s))).astype(float), self.dtype)
                        blk[off:off + take] = round8((new.astype(f) * (f(1) / f(s))).astype(float), self.dtype)
                        scales[page, h, sub] = s
                    pos, row = pos + take, row + take

    def gather(self, batch, b, head):
        """Of a sequence in 64 bits: (keys, values, positions, the values' bytes
        in the unit of the largest V scale); tokens of bad pages are absent."""
        k, v, at, units, top = [], [], [], [], 0.0
        for pos in range(0, batch.lens[b], 16):
            i = pos // self.page_size
            page = int(batch.table[b, i]) if i < batch.table.shape[1] else -1
            if not 0 <= page < self.k.shape[0]:
                continue
            sub, take = pos % self.page_size // 16, min(16, batch.lens[b] - pos)
            k.append(self.block("k", page, head, sub)[:take] * self.k_scale[page, head, sub])
            units.append(np.abs(self.block("v", page, head, sub)[:take]))
            v.append(self.block("v", page, head, sub)[:take] * self.v_scale[page, head, sub])
            top = max(top, self.v_scale[page, head, sub])
            at.append(np.arange(pos, pos + take))
        dim = self.k.shape[3]
        if not k:
            return np.zeros((0, dim)), np.zeros((0, dim)), np.zeros(0, dtype=int), np.zeros((0, dim))
        return np.concatenate(k), np.concatenate(v), np.concatenate(at), np.concatenate(units) * top


def attend(Q, plain, batch, scale, window=0, sinks=0, dtype=torch.bfloat16):
    """(O, bound): attention in 64 bits and how far the library may be from it.

    A score is a sum of dim exact products in fp32 (at most dim roundings of
    one step each, and three more for the scales); an error d of the scores
    moves a weight by a factor within exp(2d).  A weight, relative to the largest
    V scale, is rounded to fp16 once (half a step, 2^-11, or half the smallest
    step, 2^-25, where it is below fp16's normal range); its scale and the
    running maximum's factors round it by a few fp32 steps, the sums of n tokens
    by n more; the result is rounded once."""
    rows, q_heads, dim = Q.shape
    heads = plain.k.shape[1]
    group = q_heads // heads
    out, bound = np.zeros(Q.shape), np.zeros(Q.shape)
    half = EPS[dtype] / 2
    for b, (n, m) in enumerate(zip(batch.lens, batch.new)):
        r0 = int(batch.starts[b])
        for h in range(heads):
            k, v, at, unit = plain.gather(batch, b, h)
            for i in range(m):
                p = n - m + i
                sees = at <= p
                if window:
                    sees &= (p - at < window) | (at < sinks)
                if not sees.any():
                    continue
                kk, vv, uu = k[sees], v[sees], unit[sees]
                for gq in range(h * group, (h + 1) * group):
                    q = Q[r0 + i, gq]
                    s = scale * (kk @ q)
                    size = abs(scale) * (np.abs(kk) @ np.abs(q)).max()
                    d = (dim + 8) * 2.0 ** -23 * size
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    o = w @ vv
                    out[r0 + i, gq] = o
                    spread = w @ np.abs(vv)
                    rel = 2.0 ** -11 + 2 * d + (len(s) + 64) * 2.0 ** -23
                    low = 2.0 ** -25 * uu.sum(0) * w.max()
                    bound[r0 + i, gq] = 1.01 * (rel * spread + low) + half * np.abs(o) + 2.0 ** -24 * np.abs(o).max() + 1e-30
    return out, bound


def assert_close(got, want, bound, what=""):
    got = got.detach().cpu().double().numpy()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN in other places"
    err = np.abs(got - want)
    bad = ~(err <= bound) & ~nan
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside the bound; first {i}: got {got[i]!r} "
                             f"want {want[i]!r} bound {bound[i]:.3g}")
