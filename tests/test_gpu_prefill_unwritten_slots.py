"""Chunked prefill over blocks whose last slots were never written."""

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.gpu_helpers import TORCH_DTYPES
from tests.test_gpu_window import to_dev
from tests.window_helpers import cache16, window_tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("hq", [8, 10], ids=["g4", "g5"])
def test_slots_past_the_context(gpu, dtype, head_dim, window, hq):
    """Slots behind the last token (never written) may hold anything: nothing
    changes, bit for bit, with a window and without."""
    lens, new = np.array([130, 77, 33]), np.array([130, 20, 1])
    gen = np.random.default_rng(13)
    tables, nb = window_tables(lens, lens, 0, 0, gen)
    kc, vc = cache16(nb, 2, head_dim, dtype, 13, gpu)
    qs = np.concatenate([[0], np.cumsum(new)])
    q = wl.normal((int(qs[-1]), hq, head_dim), TORCH_DTYPES[dtype], 131, gpu)
    bt, cl, st = to_dev(gpu, tables, lens, qs)
    clean = pa.paged_attention_prefill_window(q, kc, vc, bt, cl, st, window, 0, 0.09)
    for bad in (float("inf"), -float("inf"), float("nan")):
        for b, n in enumerate(lens):
            for c in (kc, vc):
                c[int(tables[b, (n - 1) // 16]), :, (n - 1) % 16 + 1:] = bad
        out = pa.paged_attention_prefill_window(q, kc, vc, bt, cl, st, window, 0, 0.09)
        assert torch.equal(out, clean)
    pa.check_status()
