"""Rotary positions as dflash_paged_append_rope applies them, in float64.

Test infrastructure only (see the package docstring).  The rule is the
library's own text (include/dflash.h, "Rotary positions"); the scaling by parts
follows B. Peng et al., "YaRN: Efficient context window extension of large
language models", 2023, section 3.2.
"""

import math
from fractions import Fraction

import numpy as np


def _arctan_inverse(n, bits):
    x = (1 << bits) // n
    total, k, sign = x, 1, -1
    while x:
        x //= n * n
        k += 2
        total += sign * (x // k)
        sign = -sign
    return total


# 2 pi to 150 bits, by Machin's formula
TWO_PI = Fraction(8 * (4 * _arctan_inverse(5, 160) - _arctan_inverse(239, 160)), 1 << 160)


def frequencies(rotary_dim, theta, stretch=1.0, trained=0.0, slow=1.0, fast=4.0):
    out = []
    for j in range(rotary_dim // 2):
        w = theta ** (-2.0 * j / rotary_dim)
        if trained > 0:
            turns = trained * w / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
            out.append(keep * w + (1 - keep) * w / stretch)
        else:
            out.append(w / stretch)
    return out


def angle(position, w):
    """position * w modulo a turn, from exact rationals."""
    turns = Fraction(int(position)) * Fraction(w) / TWO_PI
    return 2 * math.pi * float(turns - math.floor(turns))


def rotate(x, positions, freq, layout, factor=1.0):
    """Rows x [n, heads, hd] turned by positions [n]; layout 0 pairs values j
    and j + rotary_dim / 2, 1 pairs 2j and 2j + 1."""
    out = np.array(x, dtype=np.float64)
    half = len(freq)
    for n, p in enumerate(positions):
        for j, w in enumerate(freq):
            a, b = (j, j + half) if layout == 0 else (2 * j, 2 * j + 1)
            t = angle(p, w)
            z = (x[n, :, a] + 1j * np.asarray(x[n, :, b], dtype=np.float64)) * factor * complex(math.cos(t), math.sin(t))
            out[n, :, a], out[n, :, b] = z.real, z.imag
    return out
