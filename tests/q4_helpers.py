"""References in 64 bits for the products with 4-bit weights and for the norms
and rotary positions, on the host.  They share no code with the library."""

from __future__ import annotations

import numpy as np
import torch

EPS = {torch.float32: 2.0 ** -23, torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}


def f64(t):
    return t.detach().cpu().double().numpy()


def weights(Q, scale, zero, group, K):
    """(M, K) float64 weights that packed codes, scales and zeros stand for."""
    q = Q.detach().cpu().numpy()
    w = np.zeros((q.shape[0], K))
    for k in range(K):
        w[:, k] = q[:, k // 2] >> 4 if k % 2 else q[:, k // 2] & 15
    at = np.arange(K) // group
    z = 8.0 if zero is None else f64(zero)[:, at]
    return (w - z) * f64(scale)[:, at]


def product(Q, scale, X, bias, zero, group, out_dtype):
    """(Y, bound).  A group's at most 128 products are exact, and so are their
    parts' where X is fp32 (three to a product); they are added in fp32, one step
    each where an adder truncates.  A matrix-core step's 32 columns may be scaled
    by themselves: K / 32 scaled sums are added, one rounding each, in at most 16
    wavefronts joined at the end; then the bias, then the rounding to Y's type by
    half a step.  The parts of an fp32 x may lose what lies below 2^-126."""
    K = X.shape[1]
    w, x = weights(Q, scale, zero, group, K), f64(X)
    y, size = x @ w.T, np.abs(x) @ np.abs(w).T
    chain = 2 * 128 * (3 if X.dtype == torch.float32 else 1) + K / 32 + 16 + 4
    fine = chain * 2.0 ** -24 * size
    if X.dtype == torch.float32:
        fine = fine + 3 * 2.0 ** -126 * np.abs(w).sum(1)[None, :]
    if bias is not None:
        b = f64(bias)
        y, fine = y + b, fine + 2.0 ** -23 * (size + np.abs(b))
    half = EPS[out_dtype] / 2 if out_dtype != torch.float32 else 0.0
    return y, fine * (1 + half) + half * np.abs(y) + TINY[out_dtype]


def rotary(x, positions, frequency, weight, eps, magnitude, interleaved, out_dtype):
    """(y, bound) of (rows, heads, dim) x.

    A norm sums dim squares in fp32 (a rounding each, halved by the root), and
    rounds the mean, the root, the quotient and two products.  A sine or cosine's
    angle, at most π, is rounded to fp32 once as a share of π (2^-24 of it), and the
    function is within 2 steps of 2^-24; the magnitude rounds it once more, and a
    value's two products and their sum a step each.  Then half a step of Y's type."""
    x = f64(x)
    rows, heads, dim = x.shape
    F = len(frequency)
    rel = 0.0
    if weight is not None:
        x = x / np.sqrt((x * x).mean(2, keepdims=True) + eps) * f64(weight)
        rel = (dim / 2 + 8) * 2.0 ** -24
    y, size = x.copy(), np.abs(x) * 0.0
    turn = np.asarray(positions, dtype=np.longdouble)[:, None] * f64(frequency).astype(np.longdouble)[None, :]
    c, s = np.cos(turn).astype(np.float64), np.sin(turn).astype(np.float64)
    for i in range(F):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + F)
        u, v = x[:, :, a], x[:, :, b]
        ci, si = c[:, i:i + 1] * magnitude, s[:, i:i + 1] * magnitude
        y[:, :, a], y[:, :, b] = u * ci - v * si, v * ci + u * si
        size[:, :, a] = size[:, :, b] = (np.abs(u) + np.abs(v)) * magnitude
    angle = np.pi * 2.0 ** -24 + 2 * 2.0 ** -24 + 3 * 2.0 ** -24
    fine = size * (angle + 2 * rel) + np.abs(x) * rel
    half = EPS[out_dtype] / 2
    return y, fine * (1 + half) + half * np.abs(y) + TINY[out_dtype]


def assert_close(got, want, bound, what=""):
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    odd = ~np.isfinite(want)
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)]), f"{what}: other infinities"
    bad = ~(np.abs(got - want) <= bound) & ~odd
    if bad.any():
        i = tuple(int(n) for n in np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside the bound; first {i}: got {got[i]!r} "
                             f"want {want[i]!r} bound {bound[i]:.3g}")
