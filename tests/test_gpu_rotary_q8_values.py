"""The rotating 8-bit decode's outputs against the oracle where a new token
joins a block whose scale stays, and where a sequence is cut over many blocks of
threads."""

import numpy as np
import pytest

from tests.test_gpu_rotary_decode import LENS, case8, check8, step8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("heads", [(8, 8), (32, 8), (10, 2), (16, 2)], ids=["g1", "g4", "g5", "g8"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
@pytest.mark.parametrize("rdim,interleaved", [(None, False), (32, True)])
def test_scales_that_stay(gpu, dtype, head_dim, heads, window, sinks, rdim, interleaved):
    lens, tables, codes, scales, q, k, v, rot, w = case8(gpu, LENS, *heads, head_dim, dtype, 40 + heads[0], window,
                                                         sinks, rdim, interleaved, 0.05)
    before = [s.clone() for s in scales]
    out, where = step8(gpu, lens, tables, codes, scales, q, k, v, rot, window, sinks)
    check8(out, where, w, rot, lens, tables, codes, scales, q, dtype, window, sinks)
    # (a block that the new token begins takes a scale of its own)
    inside = (lens > 0) & (lens % 16 != 1)
    last = tables[np.arange(len(lens)), np.maximum(lens - 1, 0) // 16][inside]
    for a, b in zip(scales, before):
        assert (a[last.tolist()] == b[last.tolist()]).float().mean() > 0.9


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [(4, 1), (16, 4), (8, 1)], ids=str)
@pytest.mark.parametrize("lens", [[40000], [3, 30000, 4], [9000, 8999, 16]], ids=str)
def test_long_sequences(gpu, dtype, heads, lens):
    lens, tables, codes, scales, q, k, v, rot, w = case8(gpu, lens, *heads, 128, dtype, 13)
    out, where = step8(gpu, lens, tables, codes, scales, q, k, v, rot, 0, 0)
    check8(out, where, w, rot, lens, tables, codes, scales, q, dtype, 0, 0)
