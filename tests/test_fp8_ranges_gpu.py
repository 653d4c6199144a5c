"""The e4m3 quantiser and product with a scale per block of 128 at the ends of
their range (needs a GPU)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import memory_bound_gemv_f32_amd as lg
from fp8_helpers import decode, quantise

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantise_rows_longer_than_a_launch(block_rows):
    """More columns than one launch's threads cover: the blocks at the cuts and
    at the end are right, and nothing else is touched."""
    K, n = (1 << 30) + 300, 1000
    x = torch.zeros(1, K, dtype=torch.float16, device="cuda")
    g = torch.Generator().manual_seed(1)
    at = [0, (1 << 29) - 512, (1 << 30) - 640]
    for a in at:
        x[0, a:a + n] = torch.randn(min(n, K - a), generator=g).to(torch.float16).cuda()
    q, s = lg.gemv_fp8_quantise(x, block_rows)
    assert q.shape == (1, K) and s.shape == (1, -(-K // 128))
    for a in at:
        want, scale = quantise(x[:, a:a + n], block_rows)
        m = n // 128 * 128 if a + n < K else n
        assert np.array_equal(decode(q[:, a:a + m]), want[:, :m])
        assert np.array_equal(s[:, a // 128:a // 128 + m // 128].cpu().numpy(), scale[:, :m // 128])
        s[0, a // 128:a // 128 + -(-n // 128)] = 2.0 ** -126
        q.view(torch.uint8)[0, a:a + 1024] = 0
    assert bool((s == 2.0 ** -126).all()) and not bool(q.view(torch.uint8).any())
