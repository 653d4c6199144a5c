"""Sizes that reach every kernel of the products with 4-bit weights: the host test holds
them against the rule, the GPU test runs them."""

import torch

FAMILIES = ("short", "staged", "few16", "few32", "few64", "tile64", "tile128", "wide64", "wide112", "wide128")
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
FAR = 1 << 22  # a pitch of X, in elements, past which tiles do not count in 32 bits


def whole(K, pad, shift):
    """Whether chunks of 128 columns and their 16-byte pieces are whole and aligned."""
    return K % 128 == 0 and pad % 16 == 0 and shift % 16 == 0


# type, family, M, K, vectors, elements between rows (of X alone where FAR), elements in
# front of the first
CASES = (
    [(t, "short", 300, 31, 40, 0, 0) for t in (F32, F16, BF16)] +
    [(F32, "staged", 150, 300, 5, 1, 0), (F32, "staged", 40, 5000, 2, 0, 3)] +
    [(t, "few16", 200, 1000, 6, 0, 0) for t in (F32, F16, BF16)] + [(F32, "few16", 40, 11000, 5, 0, 0)] +
    [(t, "few32", 4200, 300, 7, 0, 0) for t in (F32, F16, BF16)] +
    [(F32, "few64", 4200, 200, 60, 3, 1), (F32, "few64", 33000, 64, 6, FAR, 0), (F16, "few64", 2100, 500, 90, 0, 0),
     (BF16, "few64", 16400, 300, 3, 1, 0), (BF16, "few64", 33000, 64, 2, FAR, 0)] +
    # the tiles: whole chunks, ragged columns, unaligned rows
    [(F32, "tile64", 2100, K, 270, pad, shift) for K, pad, shift in ((256, 0, 0), (300, 0, 0), (128, 1, 3), (33, 0, 0))] +
    [(t, "tile64", 2000, K, 500, pad, 0) for t in (F16, BF16) for K, pad in ((256, 0), (300, 1))] +
    [(t, "tile64", 2300, K, 1100, pad, 0) for t in (F16, BF16) for K, pad in ((200, 0), (128, 1))] +
    [(F32, "tile128", 6200, K, 1000, pad, shift) for K, pad, shift in ((256, 0, 0), (77, 0, 0), (128, 3, 5))] +
    [(t, "tile128", 6200, K, 1000, pad, shift) for t in (F16, BF16) for K, pad, shift in ((256, 1, 0), (200, 0, 0), (47, 3, 5))] +
    [(t, "wide64", 2100, 256, 1100, pad, pad) for t in (F16, BF16) for pad in (0, 16)] +
    [(t, "wide112", 14336, 128, 2000, 0, 0) for t in (F16, BF16)] +
    [(t, "wide128", 4090, 384, 2030, 0, 0) for t in (F16, BF16)])
