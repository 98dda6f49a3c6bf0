"""What the tests of the grouped products share: the rows of each group as the offsets are defined to cut
them, offsets of many kinds, and e4m3 rounding in 64 bits."""

import random

import numpy as np


def spans(offsets, M):
    """(group, first row, end row) of every group: an offset counts as the largest of itself, 0 and those before
    it, and as M beyond M."""
    ends, most = [], 0
    for o in offsets:
        most = max(most, min(max(int(o), 0), M))
        ends.append(most)
    return [(e, a, b) for e, (a, b) in enumerate(zip(ends, ends[1:]))]


def even(M, E):
    return [M * e // E for e in range(E + 1)]


def ragged(M, E, seed, first=0, last=None, empty=0.3):
    """E groups over rows first .. last - 1, some of them empty."""
    rng = random.Random(seed)
    last = M if last is None else last
    cuts = sorted(rng.randint(first, last) for _ in range(E - 1))
    cuts = [first, *cuts, last]
    for i in range(1, E):
        if rng.random() < empty:
            cuts[i] = cuts[i - 1]
    return cuts


def e4m3_round(v):
    """The e4m3 value nearest to each float64 of v (magnitudes up to 464), ties to even."""
    _, exponent = np.frexp(v)
    step = np.exp2(np.maximum(exponent - 4.0, -9.0))
    return np.rint(v / step) * step


def e4m3_values():
    """The value of each of the 256 codes (NaN for 0x7F and 0xFF)."""
    code = np.arange(256)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e == 0, m * 2.0**-9, (8 + m) * 2.0 ** (e - 10.0))
    v[(code & 0x7F) == 0x7F] = np.nan
    return np.where(code & 0x80, -v, v)
