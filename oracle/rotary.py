"""Oracle of rotary positions.

TEST INFRASTRUCTURE ONLY: plain numpy, float64, from the definition: pair ``i``
of a row's first ``2 n`` columns is a complex number, which the position turns
by ``p * w_i`` and ``magnitude`` stretches; the columns behind pass through.
"""

from __future__ import annotations

import math

import numpy as np


def frequencies(rotary_dim: int, base: float, scaling: str | None = None, factor: float = 1.0,
                original_context: int = 0, low: float = 1.0, high: float = 32.0) -> np.ndarray:
    """Angle per position of every pair, one at a time."""
    out = []
    for i in range(rotary_dim // 2):
        b = base * factor ** (rotary_dim / (rotary_dim - 2)) if scaling == "base" else base
        w = math.exp(-math.log(b) * (2 * i / rotary_dim))
        if scaling == "linear":
            w = w / factor
        elif scaling == "bands":
            wavelength = 2 * math.pi / w
            turns = original_context / wavelength
            if turns <= low:
                w = w / factor
            elif turns < high:
                g = (turns - low) / (high - low)
                w = (1 - g) * (w / factor) + g * w
        out.append(w)
    return np.array(out)


def pair_columns(rotary_dim: int, interleaved: bool):
    """The two columns of each pair."""
    n = rotary_dim // 2
    if interleaved:
        return np.arange(n) * 2, np.arange(n) * 2 + 1
    return np.arange(n), np.arange(n) + n


def rotate(rows: np.ndarray, positions, w: np.ndarray, interleaved: bool = False,
           magnitude: float = 1.0):
    """``(out, size)`` of rows ``[T, H, d]``: the rotated rows, and for each
    column how much rounding errors are measured by, ``|m| (|a| + |b|)`` of its
    pair (0 in columns that pass through)."""
    out = rows.astype(np.float64).copy()
    size = np.zeros_like(out)
    first, second = pair_columns(2 * len(w), interleaved)
    with np.errstate(invalid="ignore"):
        for t, p in enumerate(positions):
            turn = magnitude * np.exp(1j * (int(p) * w))
            a, b = out[t][:, first], out[t][:, second]
            both = abs(magnitude) * (np.abs(a) + np.abs(b))
            x, y = a * turn.real - b * turn.imag, b * turn.real + a * turn.imag
            out[t][:, first], out[t][:, second] = x, y
            size[t][:, first] = size[t][:, second] = both
    return out, size
