"""Shared by the sliding-window and 8-bit cache tests: batches, inputs, and the
bound a kernel's outputs are held to."""

import numpy as np
import torch

from oracle import cache_q8 as oq
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.gpu_helpers import TORCH_DTYPES

# Half a step of each type, relative to the value: one rounding's error.
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def bound(ref, spread, size, tokens, out_type, weight_type, vmax=0.0):
    """Largest |kernel - ref| that the roundings allow.

    The kernel's out is sum w_t v_t / sum w_t rounded once to ``out_type``.
    Its scores are fp32 sums of at most 128 exact products, off by (128 + 4)
    half steps of ``size`` = scale * sum |q||k| (the 4: scale, base-2
    constant, reference, block scale); exp doubles that at most, and its own
    error is 2 steps.  A weight is rounded once to ``weight_type`` (None: kept
    in 32 bits), in the numerator and perhaps in the denominator.  Sums of
    ``tokens`` terms in fp32 add a half step each, twice (numerator and
    denominator), and as much again for rescaling and merging.  All of this is
    relative to ``spread`` = sum p_t |v_t|.  Absolute: 2^-24 for f16's subnormal
    outputs, and per token a weight under f16's smallest step, 2^-25 of the
    largest weight, times at most ``vmax`` (for the 8-bit cache 448 times the
    largest value scale, which its weights carry).
    """
    u32 = HALF_STEP["f32"]
    weight = 2 * (132 * u32 * size)[..., None] + 8 * u32 + 4 * tokens * u32
    if weight_type is not None:
        weight = weight + 2 * HALF_STEP[weight_type]
    return HALF_STEP[out_type] * np.abs(ref) * (1 + 2.0 ** -7) + weight * spread * (1 + 2.0 ** -7) \
        + 2.0 ** -24 + (tokens * 2.0 ** -25 * vmax if weight_type == "f16" else 0.0)


def assert_within(got, ref, limit, what=""):
    got = got.detach().float().cpu().numpy().astype(np.float64)
    keep = ~np.isnan(ref)
    assert np.isfinite(got[keep]).all(), f"{what}: non-finite output"
    over = np.abs(got - ref)[keep] - limit[keep]
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {over.size} outside, worst by {over.max():.3e}"


def window_tables(lens, new, window, sinks, gen, slack=3, max_blocks=None):
    """Disjoint random placement of the blocks that the newest ``new`` tokens'
    queries see; every other entry is -1 (freed)."""
    lens, new = np.asarray(lens), np.asarray(new)
    need = (lens + 15) // 16
    width = max(1, int(need.max())) if max_blocks is None else max_blocks
    col = np.arange(width)[None]
    held = col < need[:, None]
    if window:
        low = np.maximum(lens - new - window + 1, 0)[:, None]
        held &= (col * 16 < sinks) | ((col + 1) * 16 > low)
    nb = int(held.sum()) + slack
    tables = np.full((len(lens), width), -1, dtype=np.int32)
    tables[held] = gen.permutation(nb)[: int(held.sum())]
    return tables, nb


def cache16(nb, hkv, d, dtype, seed, dev):
    shape = (nb, hkv, 16, d)
    return (wl.normal(shape, TORCH_DTYPES[dtype], seed * 10 + 2, dev),
            wl.normal(shape, TORCH_DTYPES[dtype], seed * 10 + 3, dev))


def cache8(nb, hkv, d, seed, dev, spread=3):
    """Random finite codes, scales 2^-spread .. 2^spread around 2^-7 (values of
    order one)."""
    gen = np.random.default_rng(seed)
    codes = []
    for _ in range(2):
        c = oq.encode(gen.standard_normal((nb, hkv, 16, d)) * 100)
        codes.append(c)
    scales = [np.exp2(gen.integers(-7 - spread, -6 + spread, (nb, hkv))).astype(np.float32)
              for _ in range(2)]
    dev_codes = [torch.from_numpy(c).to(dev).view(torch.float8_e4m3fn) for c in codes]
    dev_scales = [torch.from_numpy(s).to(dev) for s in scales]
    return codes, scales, dev_codes, dev_scales
