"""Sizes of calls that the prompt kernel takes, with the plan that each stands for (on 152 SMs): rows of a CTA (one
row tile of 128 or two), whether its keys are cut into chunks, whether the kernel for few rows runs beside it."""
from collections import namedtuple

PromptCase = namedtuple("PromptCase", "name kv_heads group lens news window max_len rows chunks singles")

CASES = [PromptCase(*c) for c in (
    ("two tiles, whole", 8, 8, [700], [500], 0, None, 256, False, False),
    ("two tiles, window", 8, 8, [700], [500], 200, None, 256, False, False),
    # the last CTAs have 210 * 5 % 256 = 26 and 180 * 5 % 256 = 132 rows
    ("two tiles, ragged", 8, 5, [333, 290, 211] * 3, [210, 180, 210] * 3, 0, None, 256, False, True),
    ("two tiles, chunks", 1, 8, [1100], [1000], 0, None, 256, True, False),
    ("two tiles, chunks and window", 1, 8, [1500], [1000], 900, None, 256, True, False),
    ("two tiles beside single tokens", 8, 8, [900, 300, 700, 0], [700, 300, 1, 0], 0, None, 256, False, True),
    ("one tile, whole", 2, 4, [230], [180], 0, None, 128, False, False),
    ("one tile, window", 2, 4, [400], [180], 90, None, 128, False, False),
    ("one tile, chunks", 1, 2, [900], [100], 0, None, 128, True, False),
    ("one tile beside single tokens", 2, 4, [300, 90], [180, 1], 0, None, 128, False, True),
)]
BY_NAME = {c.name: c for c in CASES}
