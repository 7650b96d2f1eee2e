"""Scores of minus infinity in the rotating 16- and 32-bit decode: such a token
has no weight, wherever in the sequence it lies, whole splits of it too."""

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from tests.gpu_helpers import to_f32_numpy
from tests.test_gpu_rotary_decode import QUERY, case16, limit, reference, step16
from tests.window_helpers import assert_within

pytestmark = pytest.mark.gpu

# (a table of 63 columns is planned in splits of at most 32 blocks)
GONE = {"first": [0], "first block": range(16), "some": [0, 1, 50], "first 600": range(600),
        "all but the last": range(999)}


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("heads", [(8, 2), (16, 2)], ids=["g4", "g8"])
@pytest.mark.parametrize("gone", sorted(GONE))
def test_they_have_no_weight(gpu, dtype, heads, gone):
    lens, tables, kc, vc, q, k, v, slots, rot, w = case16(gpu, [1000, 33], *heads, 64, dtype, 13, rotary_dim=32)
    q[..., 40] = q[..., 40].abs() + 0.5                 # passes through
    for t in GONE[gone]:
        kc[int(tables[0, t // 16]), :, t % 16, 40] = -float("inf")
    out, where = step16(gpu, lens, tables, kc, vc, q, k, v, slots, rot)
    far = to_f32_numpy(kc).astype(np.float64)
    far[np.isneginf(far)] = -1e6                        # weight 0 in 64 bits
    vv = to_f32_numpy(vc)
    ref, spread, _ = reference(q, where, w, rot, far, vv, tables, lens, 0, 0, 0.125)
    clean = np.where(far == -1e6, 0.0, far)
    size = reference(q, where, w, rot, clean, vv, tables, lens, 0, 0, 0.125)[2]
    assert_within(out, ref, limit(ref, spread, size, 1000, dtype, None if dtype == "f32" else dtype,
                                  float(np.abs(vv).max()), where, w, QUERY[dtype]))
