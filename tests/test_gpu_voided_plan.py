"""A workspace as a run that gave up leaves it: the plan's signature gone, its
counters anywhere.  Runs on it do nothing and say so; a new plan makes it good
again."""

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.test_gpu_window import to_dev
from tests.window_helpers import cache16, cache8, window_tables

pytestmark = pytest.mark.gpu

WINDOW, SINKS, SCALE = 500, 4, 0.1


def refused(call, out):
    out.fill_(7.0)
    call()
    with pytest.raises(pa.PagedAttnError) as e:
        pa.check_status()
    assert e.value.status == 1
    assert (out == 7.0).all()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("head_dim", [64, 128])
def test_decode(gpu, q8, head_dim):
    lens = np.array([9000, 5, 0, 900, 16], dtype=np.int32)
    gen = np.random.default_rng(3)
    tables, nb = window_tables(lens, lens, 0, 0, gen)
    bt, cl = to_dev(gpu, tables, lens)
    q = wl.normal((5, 16, head_dim), torch.bfloat16, 5, gpu)
    out = torch.empty_like(q)
    ws = pa.alloc_window_workspace(5, 16, 4, head_dim, tables.shape[1], gpu)
    if q8:
        _, _, codes, scales = cache8(nb, 4, head_dim, 7, gpu)
        run = lambda: pa.paged_attention_decode_q8_run(q, *codes, *scales, bt, cl, WINDOW, SINKS, SCALE, ws, out=out)
    else:
        kc, vc = cache16(nb, 4, head_dim, "bf16", 7, gpu)
        run = lambda: pa.paged_attention_decode_window_run(q, kc, vc, bt, cl, WINDOW, SINKS, SCALE, ws, out=out)

    def plan():
        pa.paged_attention_decode_window_plan(cl, WINDOW, SINKS, 16, 4, head_dim, tables.shape[1], ws)

    plan()
    want = run().clone()
    ws.view(torch.int32)[0] = 0
    refused(run, out)
    ws.fill_(1)
    refused(run, out)
    plan()
    assert torch.equal(run(), want)
    assert torch.equal(run(), want)
    pa.check_status()


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("window", [0, WINDOW])
def test_prefill(gpu, head_dim, window):
    lens, new = np.array([3000, 40, 700]), np.array([70, 40, 300])
    gen = np.random.default_rng(11)
    tables, nb = window_tables(lens, lens, 0, 0, gen)
    kc, vc = cache16(nb, 4, head_dim, "bf16", 13, gpu)
    qs = np.concatenate([[0], np.cumsum(new)])
    q = wl.normal((int(qs[-1]), 16, head_dim), torch.bfloat16, 15, gpu)
    out = torch.empty_like(q)
    bt, cl, st = to_dev(gpu, tables, lens, qs)
    total = int(qs[-1])
    ws = pa.alloc_prefill_workspace(3, total, 16, 4, head_dim, gpu)

    def plan():
        pa.paged_attention_prefill_window_plan(cl, st, total, window, SINKS, 16, 4, head_dim, tables.shape[1],
                                               SCALE, torch.bfloat16, ws)

    def run():
        return pa.paged_attention_prefill_window_run(q, kc, vc, bt, cl, st, window, SINKS, SCALE, ws, out=out)

    plan()
    want = run().clone()
    ws.view(torch.int32)[3] = 0
    refused(run, out)
    ws.fill_(1)
    refused(run, out)
    plan()
    assert torch.equal(run(), want)
    assert torch.equal(run(), want)
    pa.check_status()
