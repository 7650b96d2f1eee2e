"""f16 queries near and under f16's smallest normal number, in the rotating
16-bit decode: what their rounding leaves over counts as it does for large
ones."""

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from oracle import rotary as orot
from tests.gpu_helpers import to_f32_numpy
from tests.rotary_helpers import rotary_of
from tests.test_gpu_rotary_decode import limit, reference
from tests.test_gpu_window import to_dev
from tests.window_helpers import assert_within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [(8, 8), (8, 2), (10, 2), (16, 2)], ids=str)
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("size", [2e-5, 1e-4])
def test_their_rest_counts(gpu, heads, head_dim, size):
    """Two keys along the signs of what a rotated query's rounding leaves over,
    and against them; a softmax scale that brings the scores to order one."""
    hq, hkv = heads
    gen = np.random.default_rng(7)
    rot, w = rotary_of(pa, head_dim, gpu)
    sign = np.where(gen.random((1, hq, head_dim)) < 0.5, -1.0, 1.0)
    q = torch.from_numpy(sign * size * gen.uniform(1.0, 1.2, sign.shape)).half().to(gpu)
    k = torch.zeros((1, hkv, head_dim), dtype=torch.float16, device=gpu)
    lens, where = np.array([3], dtype=np.int32), np.array([2], dtype=np.int32)
    turned, pair = orot.rotate(to_f32_numpy(q), where, w)
    rest = turned - turned.astype(np.float16).astype(np.float64)
    kc, vc = (torch.zeros((2, hkv, 16, head_dim), dtype=torch.float16, device=gpu) for _ in range(2))
    along = torch.from_numpy(np.where(rest[0, :: hq // hkv] < 0, -1.0, 1.0)).half().to(gpu)
    kc[1, :, 0], kc[1, :, 1] = along, -along
    vc[1, :, 0], vc[1, :, 1] = 1.0, -1.0
    scale = 12.0 / (head_dim * size)
    bt, cl = to_dev(gpu, np.array([[1]], dtype=np.int32), lens)
    slots = torch.tensor([16 + 2], dtype=torch.int64, device=gpu)
    ws = pa.alloc_workspace(1, hq, hkv, head_dim, 1, gpu)
    pa.paged_attention_decode_plan(cl, hq, hkv, head_dim, 1, ws)
    out = pa.paged_attention_decode_rotary_append_run(q, k, k, None, rot, slots, kc, vc, bt, cl, scale, ws)
    pa.check_status()
    ref, spread, length = reference(q, where, w, rot, to_f32_numpy(kc), to_f32_numpy(vc),
                                    np.array([[1]], dtype=np.int32), lens, 0, 0, scale)
    # a value's two parts leave 2^-22 of it, or 2^-36 where that is more: half
    # of f16's smallest step, 2^-25, under the rest's factor of 2^11
    left = 2.0 ** -22 + 2.0 ** -36 / pair.min()
    assert_within(out, ref, limit(ref, spread, length, 3, "f16", "f16", 1.0, where, w, left))
