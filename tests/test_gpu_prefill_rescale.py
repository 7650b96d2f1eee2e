"""Chunked prefill whose softmax reference has to move during a sequence, for
some rows of a warp and not for others: the accumulator is rescaled in tensor
memory by whole warps, whichever rows need it."""

import numpy as np
import pytest
import torch

import oracle.attention as oa
import pagedattention_decode_attention_gb300 as pa
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.gpu_helpers import TORCH_DTYPES, assert_attention_close, custom_batch, to_f32_numpy

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads", [(8, 8), (32, 8), (8, 1)], ids=["g1", "g4", "g8"])
def test_prefill_rows_rescale_apart(gpu, dtype, heads):
    """Keys grow along the sequence and a few rows have large queries, so that
    rows of one warp pass the rescale threshold at different tiles and some
    never do; one and two query tiles per item, several items per CTA."""
    hq, hkv = heads
    lens, new = [700, 1500, 130, 999], [260, 300, 130, 7]
    batch = custom_batch(lens, hq, hkv, 128, dtype, seed=211 + hq)
    dt = TORCH_DTYPES[dtype]
    shape = (batch.num_blocks, hkv, 16, 128)
    gen = np.random.default_rng(5)
    grow = np.ones(batch.num_blocks, dtype=np.float32)
    for b, n in enumerate(lens):
        for j in range((n + 15) // 16):
            grow[batch.block_tables[b, j]] = 2.0 ** min(3.0, j / 12)
    kc = (wl.normal(shape, torch.float32, 213, gpu) * torch.from_numpy(grow).to(gpu)[:, None, None, None]).to(dt)
    vc = wl.normal(shape, dt, 214, gpu)
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    size = np.where(gen.random((int(qs[-1]), hq, 1)) < 0.1, 4.0, 0.25).astype(np.float32)
    q = (wl.normal((int(qs[-1]), hq, 128), torch.float32, 215, gpu) * torch.from_numpy(size).to(gpu)).to(dt)
    args = [torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(gpu)
            for x in (batch.block_tables, batch.context_lens, qs)]
    out = pa.paged_attention_prefill(q, kc, vc, *args, batch.scale)
    pa.check_status()
    rows = sorted(set(range(0, int(qs[-1]), 11)))
    ref = oa.paged_attention_prefill(to_f32_numpy(q), to_f32_numpy(kc), to_f32_numpy(vc),
                                     batch.block_tables, batch.context_lens, qs, batch.scale,
                                     rows=rows)
    assert_attention_close(out, ref, dt, rows=rows)
    again = pa.paged_attention_prefill(q, kc, vc, *args, batch.scale)
    assert torch.equal(out, again)
