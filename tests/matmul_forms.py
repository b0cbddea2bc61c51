"""Which form a dense e4m3 product takes: a copy of the choice in
matmul_fp8.hip over the table of times in that file, so that a test can tell
whether its shapes still reach every form after the table has changed."""
from __future__ import annotations

import os
import re

import numpy as np

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "group_limited_routing_sigmoid_amd", "csrc", "matmul_fp8.hip")
UNITS = 256
F = np.float32


def table():
    """(rows of the table: tile height, width, times as the source has them;
    how many of them are the small tiles')."""
    text = open(SOURCE).read()
    body = re.search(r"constexpr Form kForms\[\] = \{(.*?)\};", text, re.S).group(1)
    rows = [[float(v.rstrip("f")) for v in r.split(",")] for r in re.findall(r"\{([^{}]*)\}", body)]
    forms = [(int(r[0]), int(r[1]), *(F(v) for v in r[2:])) for r in rows]
    return forms, int(re.search(r"kFormTiles = (\d+);", text).group(1))


def up(a, b):
    return -(-a // b)


def grid(M, N, form):
    """(whole rounds, tiles of the last round, pieces each is cut into)."""
    tiles = up(N, 256) * up(M, form[0])
    rest = tiles % UNITS
    split = 1
    if form[4] > 0 and rest * 2 <= UNITS:
        split = 2
    if form[5] > 0 and rest * 4 <= UNITS:
        split = 4
    return tiles // UNITS, rest, split


def choose(M, N, wide, forms, small):
    best, least = 0, None
    for i, f in enumerate(forms):
        each = f[3] if wide else f[2]
        if each < 0:
            continue
        if i < small:
            us = F(up(up(M, f[0]) * up(N, f[1]), UNITS)) * each
        else:
            full, rest, split = grid(M, N, f)
            us = F(full) * each
            if rest:
                us = us + (each if split == 1 else f[4] if split == 2 else f[5])
        if least is None or us < least:
            best, least = i, us
    return best


def case(M, N, wide, forms, small):
    """What of the code a product runs: the tile, and of the large ones whether
    there are whole rounds and how the last one's tiles are cut (0: none)."""
    i = choose(M, N, wide, forms, small)
    tile = forms[i][:2]
    if i < small:
        return (wide, *tile)
    full, rest, split = grid(M, N, forms[i])
    return (wide, *tile, full > 0, split if rest else 0)
