"""Calls of the attention over the paged 8-bit cache that reach each of its
mappings: what the host tests hold the mapping to, and what the GPU tests run
against the reference."""

from __future__ import annotations

import random

# name: lengths, new tokens (None: one each, without starts), heads, group, page size,
# window, sinks; and of the mapping (for dims 64 and 128): wavefronts that share
# rows, row tiles, whether the tokens are split
CASES = {
    "one token, four wavefronts, several chunks each": (
        [random.Random(b).randint(600, 960) for b in range(40)], None, 8, 2, 64, 0, 0, 4, 1, False),
    "one token, four wavefronts, split": (
        [random.Random(b).randint(600, 1500) for b in range(40)], None, 8, 2, 64, 0, 0, 4, 1, True),
    "one token, four wavefronts, split, windowed": (
        [random.Random(b).randint(600, 2500) for b in range(40)], None, 8, 2, 64, 1200, 70, 4, 1, True),
    "one token, eight wavefronts": ([2000, 1500], None, 4, 4, 64, 0, 0, 8, 1, True),
    "four tokens of eight heads": ([300, 90, 700], [4, 4, 4], 2, 8, 16, 0, 0, 4, 2, False),
    "four tokens of eight heads, split": ([3000, 90, 1700], [4, 4, 4], 2, 8, 64, 0, 0, 4, 2, True),
    "four tokens of eight heads, windowed": ([3000, 90, 700], [4, 4, 4], 2, 8, 64, 200, 20, 4, 2, False),
    "four tokens of eight heads, windowed, split": ([5000, 90, 2700], [4, 4, 4], 2, 8, 64, 2000, 100, 4, 2, True),
    "uneven tokens, 17 to 32 rows on average": ([900, 90, 70, 5], [60, 1, 0, 5], 2, 1, 16, 0, 0, 4, 2, False),
    "one token of 17 heads": ([700, 65, 0, 1], None, 2, 17, 32, 0, 0, 4, 2, False),
    "one token of 32 heads, split": ([2500, 700], None, 1, 32, 128, 0, 0, 4, 2, True),
    "one token of 40 heads": ([400, 65], None, 2, 40, 32, 0, 0, 1, 2, False),
    "one token of 71 heads, split": ([2500, 700], None, 1, 71, 128, 0, 0, 1, 2, True),
    "150 sequences, some of them empty": (
        [random.Random(b).randint(3, 200) for b in range(150)], [b * 7 % 4 for b in range(150)], 2, 4, 16, 0, 0, 4, 1, False),
    "90 sequences of 17 to 32 rows": (
        [random.Random(b).randint(12, 150) for b in range(90)], [b * 5 % 13 for b in range(90)], 1, 4, 16, 0, 0, 4, 2, False),
    "70 sequences of prompts": (
        [random.Random(b).randint(90, 260) for b in range(70)], [b * 11 % 90 for b in range(70)], 1, 2, 16, 0, 0, 1, 2, False),
}
