"""Scores of minus infinity (a key with an infinity in it): such a token has no
weight, wherever in the sequence it lies."""

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from oracle import windowed as ow
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.gpu_helpers import TORCH_DTYPES, to_f32_numpy
from tests.test_gpu_window import to_dev
from tests.window_helpers import assert_within, bound, cache16, window_tables

pytestmark = pytest.mark.gpu


def case(dev, dtype, d, seed, tokens):
    """K with -inf in column 0 of ``tokens`` of sequence 0, queries positive
    there: those tokens' scores are -inf."""
    lens = np.array([90, 33])
    gen = np.random.default_rng(seed)
    tables, nb = window_tables(lens, lens, 0, 0, gen)
    kc, vc = cache16(nb, 2, d, dtype, seed, dev)
    for t in tokens:
        kc[int(tables[0, t // 16]), :, t % 16, 0] = -float("inf")
    return lens, tables, kc, vc


def reference(q, kc, vc, tables, lens, qs, window, sinks, d, tokens):
    """The oracle with the tokens' weight taken out: their keys far down a
    direction of their own (finite, so the arithmetic is)."""
    k, v = to_f32_numpy(kc).astype(np.float64), to_f32_numpy(vc)
    clean = np.where(np.isinf(k), 0.0, k)
    ref, spread, size = ow.prefill(to_f32_numpy(q), clean, v, tables, lens, qs, window, sinks, d ** -0.5)
    q64 = to_f32_numpy(q).astype(np.float64)
    for row in range(int(qs[0]), int(qs[1])):              # sequence 0 by hand
        p = int(lens[0] - (qs[1] - qs[0]) + row)
        seen = [t for t in ow.visible_tokens(p, window, sinks) if t not in tokens]
        for h in range(q.shape[1]):
            g = h // (q.shape[1] // 2)
            keys = ow.gather_tokens(clean, tables[0], seen, g)
            values = ow.gather_tokens(v, tables[0], seen, g)
            ref[row, h], spread[row, h], size[row, h] = ow.attend(q64[row, h], keys, values, d ** -0.5)
    return ref, spread, size


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
@pytest.mark.parametrize("tokens", [(0,), (0, 1, 2), (50, 51), (89,)], ids=str)
def test_decode(gpu, dtype, head_dim, window, sinks, tokens):
    lens, tables, kc, vc = case(gpu, dtype, head_dim, 31, tokens)
    q = wl.normal((2, 8, head_dim), TORCH_DTYPES[dtype], 33, gpu)
    q[..., 0] = q[..., 0].abs() + 0.5
    bt, cl = to_dev(gpu, tables, lens)
    out = pa.paged_attention_decode_window(q, kc, vc, bt, cl, window, sinks, head_dim ** -0.5)
    pa.check_status()
    ref, spread, size = reference(q, kc, vc, tables, lens, [0, 1, 2], window, sinks, head_dim, tokens)
    weight = None if dtype == "f32" else dtype
    assert_within(out, ref, bound(ref, spread, size, 90, dtype, weight, float(vc.float().abs().max())))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
@pytest.mark.parametrize("tokens", [(0,), (0, 1, 2), (30, 31)], ids=str)
def test_prefill(gpu, dtype, head_dim, window, sinks, tokens):
    lens, tables, kc, vc = case(gpu, dtype, head_dim, 37, tokens)
    new = np.array([50, 33])
    qs = np.concatenate([[0], np.cumsum(new)])
    q = wl.normal((int(qs[-1]), 8, head_dim), TORCH_DTYPES[dtype], 39, gpu)
    q[..., 0] = q[..., 0].abs() + 0.5
    bt, cl, st = to_dev(gpu, tables, lens, qs)
    out = pa.paged_attention_prefill_window(q, kc, vc, bt, cl, st, window, sinks, head_dim ** -0.5)
    pa.check_status()
    ref, spread, size = reference(q, kc, vc, tables, lens, qs, window, sinks, head_dim, tokens)
    weight = None if dtype == "f32" else dtype
    assert_within(out, ref, bound(ref, spread, size, 90, dtype, weight, float(vc.float().abs().max())))
