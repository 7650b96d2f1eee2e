"""kv_append_q8 with a sequence out of order in query_start: that sequence is
skipped, every other one is stored as if it were alone."""

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from oracle import cache_q8 as oq
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.gpu_helpers import TORCH_DTYPES, to_f32_numpy
from tests.test_gpu_q8 import Mirror
from tests.test_gpu_window import to_dev
from tests.window_helpers import window_tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("starts", [
    [0, 100, 3, 108],                  # the middle one runs backwards: the third starts among the first's rows
    [0, 100, 0, 100, 0, 108],          # three whole sequences over the same rows
    [-7, 40, 90, 108],                 # rows before the first
    [0, 90, 120, 30, 108],             # past the last row, and back
    [5, 5, 5, 108, 2, 2, 60],
])
@pytest.mark.parametrize("hkv,head_dim,dtype", [(1, 64, "bf16"), (8, 64, "bf16"), (5, 128, "f32"), (2, 128, "f16")])
def test_sequences_in_order_are_stored(gpu, starts, hkv, head_dim, dtype):
    rows = 108
    n = len(starts) - 1
    lens = [130 + 3 * b for b in range(n)]
    gen = np.random.default_rng(n + hkv)
    tables, nb = window_tables(lens, lens, 0, 0, gen)
    k = wl.normal((rows, hkv, head_dim), TORCH_DTYPES[dtype], 23, gpu)
    v = wl.normal((rows, hkv, head_dim), TORCH_DTYPES[dtype], 24, gpu) * 3
    k[7, 0, 3], v[50, 0, 9] = float("inf"), float("nan")
    bt, cl, st = to_dev(gpu, tables, lens, starts)
    for _ in range(5):
        m = Mirror(nb, hkv, head_dim, 29, gpu)
        pa.kv_append_q8(k, v, *m.dcodes, *m.dscales, bt, cl, st)
        with pytest.raises(pa.PagedAttnError) as e:
            pa.check_status()
        assert e.value.status == 5
        for b in range(n):
            q0, q1 = starts[b], starts[b + 1]
            if 0 <= q0 <= q1 <= rows:
                oq.kv_append_q8(to_f32_numpy(k)[q0:q1], to_f32_numpy(v)[q0:q1], *m.codes, *m.scales,
                                tables[b:b + 1], [lens[b]], [0, q1 - q0])
        m.check()
