"""Windowed chunked prefill under a first token that takes most of the softmax:
inputs and bound are those of ``test_gpu_dominant_token.py``."""

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from tests.gpu_helpers import TORCH_DTYPES
from tests.test_gpu_dominant_token import BITS, cache, check, expected, scale_for
from tests.test_gpu_window import to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_prefill(gpu, dtype, head_dim, bits):
    """Chunks over a long context: an item's rows take all their tokens in
    turn, the first token's block first."""
    hq, hkv, window, sinks = 8, 2, 7000, 1
    lens, new = np.array([8000, 7990, 40]), np.array([90, 300, 40])
    k, v = cache(512, hkv, head_dim, 7)
    tables = np.tile(np.arange(512, dtype=np.int32), (3, 1))
    kc, vc = (torch.from_numpy(x).to(gpu, TORCH_DTYPES[dtype]) for x in (k, v))
    qs = np.concatenate([[0], np.cumsum(new)])
    q = torch.zeros((int(qs[-1]), hq, head_dim), device=gpu, dtype=TORCH_DTYPES[dtype])
    q[:, :, 0] = 1
    bt, cl, st = to_dev(gpu, tables, lens, qs)
    out = pa.paged_attention_prefill_window(q, kc, vc, bt, cl, st, window, sinks, scale_for(bits))
    pa.check_status()
    rows, seen, at = [], [], []
    for b in range(3):
        for i in (0, 1, new[b] // 2, new[b] - 1):
            p = lens[b] - new[b] + i
            t = np.arange(p + 1)
            seen.append(t[(t < sinks) | (t > p - window)])
            rows.append(qs[b] + i)
            at.append(b)
    want = expected(v, tables[at], seen, bits).repeat(4, axis=1)
    check(out[torch.tensor(rows, device=gpu)], want, 8000, bits, dtype, dtype)
