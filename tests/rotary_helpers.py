"""Shared by the tests of rotary positions."""

import numpy as np
import torch

from oracle import rotary as orot
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.gpu_helpers import TORCH_DTYPES
from tests.window_helpers import HALF_STEP

LONG = dict(base=500000.0, scaling="bands", factor=8.0, original_context=4096, low=1.0, high=4.0)

# What a kernel's cosine or sine may be off by.  The angle left after the
# nearest quarter turn is at most pi / 4 and rounded three times (integer to
# 32 bits, the constant, their product): 3 * pi / 4 half steps.  The series'
# last sum rounds once more, the terms inside it (at most 0.31 of the value,
# three roundings each) another half step, the integer's truncation and the
# series' end less than a tenth: under 4.2 half steps in all.  Then the
# magnitude's product rounds once, and x = a cos - b sin twice, each at most a
# half step of a term: 8 half steps of |m| (|a| + |b|) hold them all.
TURN_STEPS = 8.0


def angle_error(positions, w):
    """What the frequencies' own 64-bit roundings (some 2^-50 of them: exp and
    log here, pow there, the division by a turn and its 64th binary place) make
    of an angle, [T, 1, 1]."""
    p = np.abs(np.asarray(positions, dtype=np.float64))
    return (p * (np.abs(w).max() * 2.0 ** -50 + 2.0 ** -62))[:, None, None]


def rotation_error(size, positions, w):
    """Largest error of a rotated value before it is rounded to its type."""
    return size * (TURN_STEPS * HALF_STEP["f32"] + angle_error(positions, w))


def rotation_bound(ref, size, positions, w, dtype):
    """Largest |kernel - ref| of a rotated row of ``dtype``: the error in 32
    bits and one rounding (f16: or half its smallest step)."""
    e = rotation_error(size, positions, w)
    tiny = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}[dtype]
    once = np.where(size > 0, HALF_STEP[dtype] * (np.abs(ref) + e) + tiny, 0.0)
    return e + (once if dtype != "f32" else 0.0)


def projection(n, hq, hkv, d, dtype, seed, dev, pad=0):
    """q, k, v as they lie in a fused projection's output (``pad`` more columns
    behind them)."""
    x = wl.normal((n, (hq + 2 * hkv) * d + pad), TORCH_DTYPES[dtype], seed, dev)
    parts = x[:, : (hq + 2 * hkv) * d].unflatten(1, (hq + 2 * hkv, d))
    return parts.split([hq, hkv, hkv], dim=1)


def rotary_of(pa, d, dev, rotary_dim=None, interleaved=False, magnitude=1.0, **freq):
    """A ``Rotary`` and the oracle's frequencies for it."""
    r = d if rotary_dim is None else rotary_dim
    freq.setdefault("base", 10000.0)
    rot = pa.Rotary(d, dev, rotary_dim=r, interleaved=interleaved, magnitude=magnitude, **freq)
    return rot, orot.frequencies(r, **freq)


def bits(t):
    return t.contiguous().view({4: torch.int32, 2: torch.int16, 1: torch.uint8}[t.element_size()])


def same_bits(a, b):
    return torch.equal(bits(a), bits(b))
