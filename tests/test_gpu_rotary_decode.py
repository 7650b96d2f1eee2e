"""Decode steps that rotate on the way: the caches bit for bit as the append
leaves them, the output within what its roundings allow of the oracle's on
them, with the query rotated in 64 bits."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from oracle import cache_q8 as oq
from oracle import rotary as orot
from oracle import windowed as ow
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.conftest import ROOT
from tests.gpu_helpers import TORCH_DTYPES, to_f32_numpy
from tests.rotary_helpers import (LONG, TURN_STEPS, angle_error, bits, projection, rotary_of,
                                  same_bits)
from tests.test_gpu_q8 import codes_of
from tests.test_gpu_window import to_dev
from tests.window_helpers import HALF_STEP, assert_within, bound, cache8, cache16, window_tables

pytestmark = pytest.mark.gpu

LENS = [0, 1, 2, 15, 16, 17, 33, 100, 257, 530, 1999, 0]

# What is left of a rotated query's value after it is split in two parts of its
# type (its first alone in the 8-bit decode of bf16 queries, which takes f16):
# each part leaves half a step of what it is given.
QUERY = {"f32": 0.0, "f16": 2.0 ** -22, "bf16": 2.0 ** -16}
QUERY8 = {"f16": 2.0 ** -22, "bf16": 2.0 ** -11}


def reference(q, positions, w, rot, k_values, v_values, tables, lens, window, sinks, scale, k_scale=None,
              v_scale=None):
    """(out, spread, size) with the query rotated in 64 bits; ``size`` is made
    of the pairs' sums, which are no smaller than the rotated values."""
    turned, pair = orot.rotate(to_f32_numpy(q), positions, w, rot.interleaved, rot.magnitude)
    ref, spread, _ = ow.decode(turned, k_values, v_values, tables, lens, window, sinks, scale, k_scale,
                               v_scale)
    sums = np.where(pair > 0, pair, np.abs(turned))
    size = ow.decode(sums, np.abs(k_values), v_values, tables, lens, window, sinks, scale, k_scale, v_scale)[2]
    return ref, spread, size


def limit(ref, spread, size, tokens, dtype, weight, vmax, positions, w, query):
    """``bound``, and what the rotated query's own errors make of the scores:
    its cosines, its far angles, its parts (exp doubles each at most)."""
    off = TURN_STEPS * HALF_STEP["f32"] + angle_error(positions, w)[:, :, 0] + query
    more = 2 * (off * size)[..., None] * spread * (1 + 2.0 ** -7)
    return bound(ref, spread, size, tokens, dtype, weight, vmax) + more


def case16(dev, lens, hq, hkv, d, dtype, seed, rotary_dim=None, interleaved=False, pad=8, **freq):
    gen = np.random.default_rng(seed)
    lens = np.asarray(lens, dtype=np.int32)
    tables, nb = window_tables(np.maximum(lens, 1), lens, 0, 0, gen)
    kc, vc = cache16(nb, hkv, d, dtype, seed, dev)
    q, k, v = projection(len(lens), hq, hkv, d, dtype, seed + 1, dev, pad)
    last = np.maximum(lens - 1, 0)
    slots = tables[np.arange(len(lens)), last // 16].astype(np.int64) * 16 + last % 16
    rot, w = rotary_of(pa, d, dev, rotary_dim, interleaved, **freq)
    return lens, tables, kc, vc, q, k, v, slots, rot, w


def step16(dev, lens, tables, kc, vc, q, k, v, slots, rot, positions=None):
    """One launch's output, after checking the caches against rotary_kv_append's."""
    d, (hq, hkv) = q.shape[2], (q.shape[1], k.shape[1])
    bt, cl = to_dev(dev, tables, lens)
    ds = torch.from_numpy(slots).to(dev)
    where = (lens - 1).astype(np.int32) if positions is None else np.asarray(positions, dtype=np.int32)
    pos = torch.from_numpy(where).to(dev)
    kw, vw = kc.clone(), vc.clone()
    pa.rotary_kv_append(None, k, v, pos, rot, kw, vw, ds)
    ws = pa.alloc_workspace(len(lens), hq, hkv, d, tables.shape[1], dev)
    pa.paged_attention_decode_plan(cl, hq, hkv, d, tables.shape[1], ws)
    scale = d ** -0.5
    out = pa.paged_attention_decode_rotary_append_run(q, k, v, None if positions is None else pos, rot, ds, kc, vc,
                                                      bt, cl, scale, ws)
    again = torch.empty_like(out)
    op = pa.prepare_decode_rotary_append_run(q, k, v, pos, rot, ds, kc, vc, bt, cl, scale, ws, again)
    op()
    pa.check_status()
    assert same_bits(kc, kw) and same_bits(vc, vw)
    assert same_bits(again, out)
    return out, where


def check16(out, where, w, rot, lens, tables, kc, vc, q, dtype):
    ref, spread, size = reference(q, where, w, rot, to_f32_numpy(kc), to_f32_numpy(vc), tables, lens, 0, 0,
                                  q.shape[2] ** -0.5)
    assert_within(out, ref, limit(ref, spread, size, int(lens.max()), dtype, None if dtype == "f32" else dtype,
                                  float(vc.float().abs().max()), where, w, QUERY[dtype]))
    assert (out[torch.from_numpy(lens == 0)] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("heads", [(8, 8), (32, 8), (10, 2), (16, 2)], ids=["g1", "g4", "g5", "g8"])
@pytest.mark.parametrize("rdim,interleaved", [(None, False), (None, True), (48, False), (32, True)])
def test_matches_oracle(gpu, dtype, head_dim, heads, rdim, interleaved):
    lens, tables, kc, vc, q, k, v, slots, rot, w = case16(gpu, LENS, *heads, head_dim, dtype, 40 + heads[0],
                                                          rdim, interleaved, magnitude=1.1 if rdim else 1.0)
    out, where = step16(gpu, lens, tables, kc, vc, q, k, v, slots, rot)
    check16(out, where, w, rot, lens, tables, kc, vc, q, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_given_positions_and_long_contexts(gpu, dtype):
    """Positions of the caller's (a stretched context, far and negative ones)."""
    lens, tables, kc, vc, q, k, v, slots, rot, w = case16(gpu, LENS, 32, 8, 128, dtype, 7, **LONG)
    positions = [5, 0, 131071, 2 ** 31 - 1, -7, 30, 31, 65536, 1, 2, 999999, -2 ** 31]
    out, where = step16(gpu, lens, tables, kc, vc, q, k, v, slots, rot, positions)
    check16(out, where, w, rot, lens, tables, kc, vc, q, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_tokens_that_are_not_stored(gpu, dtype):
    """A negative slot: the cache is attended as it is, the query rotated."""
    lens, tables, kc, vc, q, k, v, slots, rot, w = case16(gpu, LENS, 32, 8, 128, dtype, 9)
    slots[[2, 5, 7, 11]] = -1
    out, where = step16(gpu, lens, tables, kc, vc, q, k, v, slots, rot)
    check16(out, where, w, rot, lens, tables, kc, vc, q, dtype)


def test_bad_slots_are_reported(gpu):
    lens, tables, kc, vc, q, k, v, slots, rot, w = case16(gpu, [40, 40, 40, 0], 8, 2, 128, "bf16", 9)
    bt, cl = to_dev(gpu, tables, lens)
    slots[1], slots[3] = kc.shape[0] * 16, 1 << 40
    kw, vw = kc.clone(), vc.clone()
    good = slots.copy()
    good[[1, 3]] = -1
    pa.rotary_kv_append(None, k, v, cl - 1, rot, kw, vw, torch.from_numpy(good).to(gpu))
    ws = pa.alloc_workspace(4, 8, 2, 128, tables.shape[1], gpu)
    pa.paged_attention_decode_plan(cl, 8, 2, 128, tables.shape[1], ws)
    pa.paged_attention_decode_rotary_append_run(q, k, v, None, rot, torch.from_numpy(slots).to(gpu), kc, vc, bt,
                                                cl, 0.1, ws)
    with pytest.raises(pa.PagedAttnError) as e:
        pa.check_status()
    assert e.value.status == 5
    assert same_bits(kc, kw) and same_bits(vc, vw)


def test_a_run_needs_its_plan(gpu):
    lens, tables, kc, vc, q, k, v, slots, rot, w = case16(gpu, [40, 300], 8, 2, 128, "bf16", 9)
    bt, cl = to_dev(gpu, tables, lens)
    ws = torch.zeros(pa.workspace_size(2, 8, 2, 128, tables.shape[1]), dtype=torch.uint8, device=gpu)
    out = torch.full_like(q, 7.0, memory_format=torch.contiguous_format)
    kw = kc.clone()
    pa.paged_attention_decode_rotary_append_run(q, k, v, None, rot, torch.from_numpy(slots).to(gpu), kc, vc, bt,
                                                cl, 0.1, ws, out=out)
    with pytest.raises(pa.PagedAttnError) as e:
        pa.check_status()
    assert e.value.status == 1
    assert (out == 7).all() and same_bits(kc, kw)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
def test_long_and_many_sequences(gpu, dtype, head_dim):
    """Splits merged over warps, and more sequences than warps."""
    gen = np.random.default_rng(5)
    for lens, rows in (([20011, 3, 7777], None), (list(gen.integers(0, 200, 700)), range(0, 700, 23))):
        lens, tables, kc, vc, q, k, v, slots, rot, w = case16(gpu, lens, 8, 2, head_dim, dtype, 11)
        out, where = step16(gpu, lens, tables, kc, vc, q, k, v, slots, rot)
        rows = list(range(len(lens)) if rows is None else rows)
        at = torch.tensor(rows, device=gpu)
        check16(out[at], where[rows], w, rot, lens[rows], tables[rows], kc, vc, q[at], dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_a_token_that_takes_almost_everything(gpu, dtype):
    """One key far along the query, thousands of others under it: their share
    is small but theirs."""
    n = 6000
    lens, tables, kc, vc, q, k, v, slots, rot, w = case16(gpu, [n], 8, 2, 128, dtype, 13)
    where = np.array([n - 1], dtype=np.int32)
    turned, _ = orot.rotate(to_f32_numpy(q), where, w)
    kc.mul_(0.05)
    for g in range(2):
        row = turned[0, 4 * g]
        kc[int(tables[0, 0]), g, 3] = torch.from_numpy(row * (13.0 / (128 ** -0.5 * (row @ row)))).to(kc.dtype).to(gpu)
    out, where = step16(gpu, lens, tables, kc, vc, q, k, v, slots, rot)
    ref, spread, size = reference(q, where, w, rot, to_f32_numpy(kc), to_f32_numpy(vc), tables, lens, 0, 0,
                                  128 ** -0.5)
    # (f16 weights are lifted by 2^7: half of f16's smallest step lies 2^-32 under the largest)
    assert_within(out, ref, limit(ref, spread, size, n, dtype, dtype, float(vc.float().abs().max()) * 2.0 ** -7,
                                  where, w, QUERY[dtype]))


def test_scores_of_minus_infinity(gpu):
    """Keys with an infinity that the rotated query meets with one sign: no
    weight, wherever they lie (the first block whole)."""
    lens, tables, kc, vc, q, k, v, slots, rot, w = case16(gpu, [90, 33], 8, 2, 64, "bf16", 13, rotary_dim=32)
    q[..., 40] = q[..., 40].abs() + 0.5                 # passes through
    gone = list(range(16)) + [50]
    for t in gone:
        kc[int(tables[0, t // 16]), :, t % 16, 40] = -float("inf")
    out, where = step16(gpu, lens, tables, kc, vc, q, k, v, slots, rot)
    far = to_f32_numpy(kc).astype(np.float64)
    far[np.isneginf(far)] = -1e6                        # weight 0 in 64 bits
    ref, spread, _ = reference(q, where, w, rot, far, to_f32_numpy(vc), tables, lens, 0, 0, 0.125)
    clean = np.where(far == -1e6, 0.0, far)
    size = reference(q, where, w, rot, clean, to_f32_numpy(vc), tables, lens, 0, 0, 0.125)[2]
    assert_within(out, ref, limit(ref, spread, size, 90, "bf16", "bf16", 0.0, where, w, QUERY["bf16"]))


@pytest.mark.parametrize("heads", [(1, 1), (7, 1), (8, 2)], ids=str)
def test_rows_that_repeat(gpu, heads):
    """A stride of zero: every sequence with the same query, key and value."""
    lens, tables, kc, vc, q, k, v, slots, rot, w = case16(gpu, [40, 1, 300, 17], *heads, 128, "bf16", 13)
    one = [t[:1].expand(4, -1, -1) for t in (q, k, v)]
    kw, vw = kc.clone(), vc.clone()
    want, _ = step16(gpu, lens, tables, kw, vw, *(t.contiguous() for t in one), slots, rot)
    got, where = step16(gpu, lens, tables, kc, vc, *one, slots, rot)
    assert same_bits(got, want) and same_bits(kc, kw)
    check16(got, where, w, rot, lens, tables, kc, vc, one[0], "bf16")


def test_unwritten_slots_may_hold_anything(gpu):
    """NaN and infinities behind the last token, and in the new token's slot
    before it is written."""
    lens, tables, kc, vc, q, k, v, slots, rot, w = case16(gpu, [1, 17, 31, 40], 8, 2, 128, "f16", 13)
    for b, n in enumerate(lens):
        for t in range(n - 1, (n + 15) // 16 * 16):
            for c, x in ((kc, float("nan")), (vc, float("inf"))):
                c[int(tables[b, t // 16]), :, t % 16] = x
    clean_k, clean_v = kc.nan_to_num(0, 0, 0), vc.nan_to_num(0, 0, 0)
    want, _ = step16(gpu, lens, tables, clean_k, clean_v, q, k, v, slots, rot)
    bt, cl = to_dev(gpu, tables, lens)
    ws = pa.alloc_workspace(4, 8, 2, 128, tables.shape[1], gpu)
    pa.paged_attention_decode_plan(cl, 8, 2, 128, tables.shape[1], ws)
    got = pa.paged_attention_decode_rotary_append_run(q, k, v, None, rot, torch.from_numpy(slots).to(gpu), kc, vc,
                                                      bt, cl, 128 ** -0.5, ws)
    pa.check_status()
    assert same_bits(got, want)


# ---------------------------------------------------------------- 8-bit cache
def case8(dev, lens, hq, hkv, d, dtype, seed, window=0, sinks=0, rotary_dim=None, interleaved=False, size=1.0,
          **freq):
    gen = np.random.default_rng(seed)
    lens = np.asarray(lens, dtype=np.int32)
    tables, nb = window_tables(lens, [1] * len(lens), window, sinks, gen)
    _, _, codes, scales = cache8(nb, hkv, d, seed, dev)
    q, k, v = projection(len(lens), hq, hkv, d, dtype, seed + 1, dev, 8)
    k *= size
    v *= size
    rot, w = rotary_of(pa, d, dev, rotary_dim, interleaved, **freq)
    return lens, tables, codes, scales, q, k, v, rot, w


def step8(dev, lens, tables, codes, scales, q, k, v, rot, window, sinks, positions=None):
    d, (hq, hkv) = q.shape[2], (q.shape[1], k.shape[1])
    where = (lens - 1).astype(np.int32) if positions is None else np.asarray(positions, dtype=np.int32)
    has = lens > 0
    starts = np.concatenate([[0], np.cumsum(has)])
    bt, cl, st = to_dev(dev, tables, lens, starts)
    pos = torch.from_numpy(where).to(dev)
    keep = torch.from_numpy(np.flatnonzero(has)).to(dev)
    want = [t.clone() for t in (*codes, *scales)]
    pa.rotary_kv_append_q8(None, k[keep], v[keep], pos[keep], rot, *want, bt, cl, st)
    ws = pa.alloc_window_workspace(len(lens), hq, hkv, d, tables.shape[1], dev)
    pa.paged_attention_decode_window_plan(cl, window, sinks, hq, hkv, d, tables.shape[1], ws)
    out = pa.paged_attention_decode_q8_rotary_append_run(q, k, v, None if positions is None else pos, rot, *codes,
                                                         *scales, bt, cl, window, sinks, d ** -0.5, ws)
    again = torch.empty_like(out)
    op = pa.prepare_decode_q8_rotary_append_run(q, k, v, pos, rot, *codes, *scales, bt, cl, window, sinks,
                                                d ** -0.5, ws, again)
    op()
    pa.check_status()
    for a, b in zip((*codes, *scales), want):
        assert same_bits(a, b)
    assert same_bits(again, out)
    return out, where


def check8(out, where, w, rot, lens, tables, codes, scales, q, dtype, window, sinks):
    d = q.shape[2]
    kv, vv = (oq.decode(codes_of(c)) for c in codes)
    ks, vs = (s.cpu().numpy() for s in scales)
    ref, spread, size = reference(q, where, w, rot, kv, vv, tables, lens, window, sinks, d ** -0.5, ks, vs)
    tokens = min(int(lens.max()), window + sinks) if window else int(lens.max())
    assert_within(out, ref, limit(ref, spread, size, tokens, dtype, "f16", 448.0 * float(vs.max()), where, w,
                                  QUERY8[dtype]))
    assert (out[torch.from_numpy(lens == 0)] == 0).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("heads", [(8, 8), (32, 8), (10, 2), (16, 2)], ids=["g1", "g4", "g5", "g8"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 4)])
@pytest.mark.parametrize("rdim,interleaved", [(None, False), (None, True), (48, False), (32, True)])
def test_q8_matches_oracle(gpu, dtype, head_dim, heads, window, sinks, rdim, interleaved):
    for size in (0.05, 40.0):           # scales that stay and that grow
        case = case8(gpu, LENS, *heads, head_dim, dtype, 40 + heads[0], window, sinks, rdim, interleaved, size,
                     magnitude=1.1 if rdim else 1.0)
        lens, tables, codes, scales, q, k, v, rot, w = case
        out, where = step8(gpu, lens, tables, codes, scales, q, k, v, rot, window, sinks)
    check8(out, where, w, rot, lens, tables, codes, scales, q, dtype, window, sinks)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_q8_given_positions(gpu, dtype):
    lens, tables, codes, scales, q, k, v, rot, w = case8(gpu, LENS, 32, 8, 128, dtype, 7, **LONG)
    positions = [5, 0, 131071, 2 ** 31 - 1, -7, 30, 31, 65536, 1, 2, 999999, -2 ** 31]
    out, where = step8(gpu, lens, tables, codes, scales, q, k, v, rot, 0, 0, positions)
    check8(out, where, w, rot, lens, tables, codes, scales, q, dtype, 0, 0)


@pytest.mark.parametrize("dtype,size", [("bf16", 1e30), ("bf16", 1e-30), ("f16", 60000.0), ("f16", 1e-6)])
def test_q8_queries_of_any_size(gpu, dtype, size):
    """Rows of any size keep their direction (the softmax scale takes the size
    out); f16 rows past f16's range once rotated too."""
    lens, tables, codes, scales, q, k, v, rot, w = case8(gpu, [40, 130], 8, 2, 128, dtype, 7)
    unit = q / q.float().abs().amax(-1, keepdim=True)
    big = (unit.float() * size).to(q.dtype)
    bt, cl = to_dev(gpu, tables, lens)
    ws = pa.alloc_window_workspace(2, 8, 2, 128, tables.shape[1], gpu)
    pa.paged_attention_decode_window_plan(cl, 0, 0, 8, 2, 128, tables.shape[1], ws)
    out = pa.paged_attention_decode_q8_rotary_append_run(big, k, v, None, rot, *codes, *scales, bt, cl, 0, 0,
                                                         2.0 / size, ws)
    pa.check_status()
    kv, vv = (oq.decode(codes_of(c)) for c in codes)
    ks, vs = (s.cpu().numpy() for s in scales)
    where = lens - 1
    ref, spread, length = reference(big, where, w, rot, kv, vv, tables, lens, 0, 0, 2.0 / size, ks, vs)
    assert_within(out, ref, limit(ref, spread, length, 130, dtype, "f16", 448.0 * float(vs.max()), where, w,
                                  QUERY8[dtype]))


def test_q8_batches_of_every_size(gpu):
    gen = np.random.default_rng(11)
    for lens in ([5], [1] * 300, [40000], list(gen.integers(0, 90, 513)), [3, 30000, 4]):
        lens, tables, codes, scales, q, k, v, rot, w = case8(gpu, lens, 16, 4, 128, "bf16", 13)
        out, where = step8(gpu, lens, tables, codes, scales, q, k, v, rot, 0, 0)
        if len(lens) > 300:
            rows = list(range(0, 513, 31))
            at = torch.tensor(rows, device=gpu)
            check8(out[at], where[rows], w, rot, lens[rows], tables[rows], codes, scales, q[at], "bf16", 0, 0)
        elif lens.max() < 1000:
            check8(out, where, w, rot, lens, tables, codes, scales, q, "bf16", 0, 0)


def test_q8_special_values(gpu):
    """Zeros, infinities and NaN among the new rows store what the append
    stores."""
    lens, tables, codes, scales, q, k, v, rot, w = case8(gpu, [1, 1, 17, 18, 40, 31], 8, 2, 64, "bf16", 5)
    k[0], v[1], k[2, 0, 3], v[3, 1, 60] = 0, 0, float("inf"), float("nan")
    k[4], v[5] = float("nan"), -float("inf")
    bt, cl, st = to_dev(gpu, tables, lens, range(7))
    want = [t.clone() for t in (*codes, *scales)]
    pa.rotary_kv_append_q8(None, k, v, None, rot, *want, bt, cl, st)
    ws = pa.alloc_window_workspace(6, 8, 2, 64, tables.shape[1], gpu)
    pa.paged_attention_decode_window_plan(cl, 0, 0, 8, 2, 64, tables.shape[1], ws)
    pa.paged_attention_decode_q8_rotary_append_run(q, k, v, None, rot, *codes, *scales, bt, cl, 0, 0, 0.125, ws)
    pa.check_status()
    for i in range(2):
        nan = (bits(want[i]) & 0x7F) == 0x7F
        assert torch.equal(nan, (bits(codes[i]) & 0x7F) == 0x7F)
        assert torch.equal(bits(codes[i])[~nan], bits(want[i])[~nan])
        assert same_bits(scales[i], want[2 + i])


def test_q8_bad_block_and_no_plan(gpu):
    lens, tables, codes, scales, q, k, v, rot, w = case8(gpu, [20, 33, 48], 8, 2, 128, "bf16", 5)
    dirty = tables.copy()
    dirty[1, 2] = 1 << 20
    bt, cl = to_dev(gpu, dirty, lens)
    want = [t.clone() for t in (*codes, *scales)]
    two, st = to_dev(gpu, [lens[0], lens[2]], [0, 1, 2])
    keep = torch.tensor([0, 2], device=gpu)
    pa.rotary_kv_append_q8(None, k[keep], v[keep], None, rot, *want, bt[keep].contiguous(), two, st)
    ws = pa.alloc_window_workspace(3, 8, 2, 128, 3, gpu)
    ws.zero_()
    out = torch.full((3, 8, 128), 7.0, dtype=q.dtype, device=gpu)
    run = lambda: pa.paged_attention_decode_q8_rotary_append_run(
        q, k, v, None, rot, *codes, *scales, bt, cl, 0, 0, 0.1, ws, out=out)
    before = [t.clone() for t in (*codes, *scales)]
    run()
    with pytest.raises(pa.PagedAttnError) as e:
        pa.check_status()
    assert e.value.status == 1 and (out == 7).all()
    for a, b in zip((*codes, *scales), before):
        assert same_bits(a, b)
    pa.paged_attention_decode_window_plan(cl, 0, 0, 8, 2, 128, 3, ws)
    run()
    with pytest.raises(pa.PagedAttnError) as e:
        pa.check_status()
    assert e.value.status == 5
    for a, b in zip((*codes, *scales), want):
        assert same_bits(a, b)


# ------------------------------------------------------------------- together
@pytest.mark.parametrize("q8", [False, True])
def test_streams_and_graphs(gpu, q8):
    """A step on another stream, two steps at once with workspaces of their
    own, and one captured and replayed."""
    def make(seed):
        if q8:
            lens, tables, codes, scales, q, k, v, rot, w = case8(gpu, LENS, 32, 8, 128, "bf16", seed)
            cache = [*codes, *scales]
        else:
            lens, tables, kc, vc, q, k, v, slots, rot, w = case16(gpu, LENS, 32, 8, 128, "bf16", seed)
            cache = [kc, vc]
        bt, cl = to_dev(gpu, tables, lens)
        mb = tables.shape[1]
        if q8:
            ws = pa.alloc_window_workspace(len(lens), 32, 8, 128, mb, gpu)
            plan = lambda **s: pa.paged_attention_decode_window_plan(cl, 0, 0, 32, 8, 128, mb, ws, **s)
            run = lambda **s: pa.paged_attention_decode_q8_rotary_append_run(
                q, k, v, None, rot, *cache, bt, cl, 0, 0, 0.1, ws, **s)
        else:
            ds = torch.from_numpy(slots).to(gpu)
            ws = pa.alloc_workspace(len(lens), 32, 8, 128, mb, gpu)
            plan = lambda **s: pa.paged_attention_decode_plan(cl, 32, 8, 128, mb, ws, **s)
            run = lambda **s: pa.paged_attention_decode_rotary_append_run(
                q, k, v, None, rot, ds, *cache, bt, cl, 0.1, ws, **s)
        return plan, run, q

    first, second = make(3), make(4)
    want = []
    for plan, run, _ in (first, second):
        plan()
        want.append(run().clone())
    streams = [torch.cuda.Stream(gpu) for _ in range(2)]
    main = torch.cuda.current_stream(gpu)
    for _ in range(5):
        got = []
        for s, (plan, run, _) in zip(streams, (first, second)):
            s.wait_stream(main)
            plan(stream=s)
            got.append(run(stream=s))
        for s in streams:
            main.wait_stream(s)
        assert same_bits(got[0], want[0]) and same_bits(got[1], want[1])
    plan, run, q = first
    out = torch.empty(q.shape, dtype=q.dtype, device=gpu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan()
        run(out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert same_bits(out, want[0])
    pa.check_status()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_a_prompt_and_its_answer(gpu, dtype):
    """As a server uses them: prompt chunks rotated into the cache and attended
    (prefill), then single tokens, each step one launch; every output against
    attention over the whole rotated sequence in 64 bits."""
    d, hq, hkv, scale = 128, 8, 2, 128 ** -0.5
    rot, w = rotary_of(pa, d, gpu, **LONG)
    total, prompt = [150, 61], [[70, 60], [30, 20]]
    gen = np.random.default_rng(3)
    tables, nb = window_tables(total, total, 0, 0, gen)
    kc, vc = cache16(nb, hkv, d, dtype, 5, gpu)
    bt = to_dev(gpu, tables)[0]
    rows = [projection(n, hq, hkv, d, dtype, 9 + b, gpu) for b, n in enumerate(total)]
    done = [0, 0]
    outs = [[], []]

    def slots_of(b, places):
        return tables[b, places // 16].astype(np.int64) * 16 + places % 16

    for step in range(2):                                       # two chunks of each prompt
        new = [prompt[b][step] for b in range(2)]
        q, k, v = (torch.cat([rows[b][i][done[b]: done[b] + new[b]] for b in range(2)]) for i in range(3))
        where = np.concatenate([np.arange(done[b], done[b] + new[b]) for b in range(2)])
        slots = np.concatenate([slots_of(b, np.arange(done[b], done[b] + new[b])) for b in range(2)])
        done = [done[b] + new[b] for b in range(2)]
        cl, qs, pos = to_dev(gpu, done, [0, new[0], sum(new)], where)
        turned = pa.rotary_kv_append(q, k, v, pos, rot, kc, vc, torch.from_numpy(slots).to(gpu))
        out = pa.paged_attention_prefill(turned, kc, vc, bt, cl, qs, scale)
        outs[0].append(out[: new[0]])
        outs[1].append(out[new[0]:])
    ws = pa.alloc_workspace(2, hq, hkv, d, tables.shape[1], gpu)
    while done[0] < total[0]:                                   # single tokens; the short one ends first
        live = [b for b in range(2) if done[b] < total[b]]
        q, k, v = (torch.cat([rows[b][i][min(done[b], total[b] - 1)][None] for b in range(2)]) for i in range(3))
        done = [done[b] + (b in live) for b in range(2)]
        slots = [slots_of(b, np.array([done[b] - 1]))[0] if b in live else -1 for b in range(2)]
        cl = to_dev(gpu, done)[0]
        pa.paged_attention_decode_plan(cl, hq, hkv, d, tables.shape[1], ws)
        out = pa.paged_attention_decode_rotary_append_run(q, k, v, None, rot, torch.tensor(slots, device=gpu), kc,
                                                          vc, bt, cl, scale, ws)
        for b in live:
            outs[b].append(out[b: b + 1])
    pa.check_status()
    kh, vh = to_f32_numpy(kc).astype(np.float64), to_f32_numpy(vc)
    half = HALF_STEP[dtype]
    for b in range(2):
        n = total[b]
        got = torch.cat(outs[b])
        places = np.arange(n)
        turned, pair = orot.rotate(to_f32_numpy(rows[b][0]), places, w)
        keys, ksize = orot.rotate(to_f32_numpy(rows[b][1]), places, w)
        # the cache holds the rotated keys, once rounded
        held = np.stack([ow.gather_tokens(kh, tables[b], range(n), g) for g in range(hkv)], 1)
        room = ksize * (TURN_STEPS * HALF_STEP["f32"] + angle_error(places, w))
        assert (np.abs(held - keys) <= room + half * (np.abs(keys) + room) + 2.0 ** -25).all()
        ref, spread, _ = ow.prefill(turned, kh, vh, tables[b: b + 1], [n], [0, n], 0, 0, scale)
        size = ow.prefill(pair, np.abs(kh), vh, tables[b: b + 1], [n], [0, n], 0, 0, scale)[2]
        # the prompt's queries are stored rotated, in their type: half a step
        # more of the scores' size (the answer's are not, but may be)
        weight = None if dtype == "f32" else dtype
        assert_within(got, ref, limit(ref, spread, size, n, dtype, weight, float(vc.float().abs().max()), places, w,
                                      half))


def test_tuned_processes(gpu):
    """The rotating decode under other ring, split and CTA settings."""
    for env in (dict(PA_DECODE_WARPS="4", PA_DECODE_CTAS_PER_SM="2"), dict(PA_DECODE_MAX_STAGES="1"),
                dict(PA_DECODE_TAIL_WAVES="0", PA_DECODE_SPLIT_BLOCKS="16")):
        res = subprocess.run([sys.executable, "-m", "tests.rotary_child"], cwd=ROOT, env={**os.environ, **env},
                             capture_output=True, text=True, timeout=300)
        assert res.returncode == 0, res.stdout + res.stderr
