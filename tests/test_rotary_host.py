"""The frequencies of rotary positions against their rule, pair by pair, in 64 bits
(no GPU)."""

from __future__ import annotations

import math

import numpy as np
import pytest

import memory_bound_gemv_f32_amd as lg


def pair_that_turns(times, dim, base, original):
    """The i, not whole, whose frequency base^(-2i/dim) turns so often within `original`."""
    return dim / 2 * math.log(original / (2 * math.pi * times), base)


@pytest.mark.parametrize("dim", [2, 32, 64, 96, 128, 256])
@pytest.mark.parametrize("base", [500.0, 10000.0, 500000.0, 1e7])
def test_every_pair_of_a_stretched_context(dim, base):
    """Divided, kept or between by its own number of turns, for contexts that are short
    or long beside the slowest pair's turn, and linear in i between."""
    for original in (3, 5, 100, 1000, 4096, 8192, 32768, 131072, 1 << 20, 1 << 24):
        for factor, fast, slow in ((4.0, 32.0, 1.0), (40.0, 32.0, 1.0), (1.5, 8.0, 2.0)):
            f, magnitude = lg.rotary_frequencies(dim, base, factor=factor, original=original, fast=fast, slow=slow, device="cpu")
            assert f.shape == (dim // 2,) and abs(magnitude - (1 + 0.1 * math.log(factor))) < 1e-12
            low = math.floor(pair_that_turns(fast, dim, base, original))
            high = math.ceil(pair_that_turns(slow, dim, base, original))
            for i in range(dim // 2):
                plain = base ** (-2.0 * i / dim)
                turns = original * plain / (2 * math.pi)
                share = min(max((i - low) / (high - low), 0.0), 1.0)
                want = plain * (1 - share) + plain / factor * share
                what = (original, factor, i, turns)
                assert abs(float(f[i]) - want) <= 2.0 ** -23 * want, what
                if turns < slow * (1 - 1e-9):
                    assert abs(float(f[i]) - plain / factor) <= 2.0 ** -23 * plain, what
                if turns > fast * (1 + 1e-9):
                    assert abs(float(f[i]) - plain) <= 2.0 ** -23 * plain, what


def test_the_last_pair_of_a_long_context():
    """128 values, base 10000, a context of 131072: the last pair turns 2.4 times,
    which is between, 18 of 25 pairs past the one that turns 32 times."""
    f, _ = lg.rotary_frequencies(128, 10000.0, factor=4.0, original=131072, device="cpu")
    ratio = float(f[63]) / 10000.0 ** (-126 / 128)
    assert abs(ratio - (1 - 0.75 * 18 / 25)) < 1e-6


def test_a_context_shorter_than_any_turn():
    """Every pair turns less than once: all are divided."""
    f, _ = lg.rotary_frequencies(64, 10000.0, factor=8.0, original=4, device="cpu")
    assert np.allclose(f.double().numpy(), 10000.0 ** (-np.arange(32) / 32) / 8, rtol=2.0 ** -23)


def test_no_values():
    f, magnitude = lg.rotary_frequencies(0, 10000.0, factor=2.0, original=4096, device="cpu")
    assert f.shape == (0,) and magnitude > 1
