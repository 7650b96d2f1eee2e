"""Sliding-window attention on the GPU (decode and chunked prefill) against the
64-bit oracle, over lengths, windows, first tokens, groups and types where it
can go wrong.  Bounds come from ``tests/window_helpers.py``."""

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from oracle import windowed as ow
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.gpu_helpers import TORCH_DTYPES, to_f32_numpy
from tests.window_helpers import assert_within, bound, cache16, window_tables

pytestmark = pytest.mark.gpu

LENS = [0, 1, 15, 16, 17, 33, 100, 257, 530, 1999]


def to_dev(dev, *arrays):
    return [torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev) for a in arrays]


def decode_case(dev, lens, hq, hkv, d, dtype, window, sinks, seed, max_blocks=None):
    gen = np.random.default_rng(seed)
    lens = np.asarray(lens, dtype=np.int32)
    tables, nb = window_tables(lens, [1] * len(lens), window, sinks, gen, max_blocks=max_blocks)
    kc, vc = cache16(nb, hkv, d, dtype, seed, dev)
    q = wl.normal((len(lens), hq, d), TORCH_DTYPES[dtype], seed * 10 + 1, dev)
    return q, kc, vc, tables, lens


def check_decode(out, q, kc, vc, tables, lens, window, sinks, dtype, rows=None, scale=None):
    d = q.shape[2]
    ref, spread, size = ow.decode(to_f32_numpy(q), to_f32_numpy(kc), to_f32_numpy(vc), tables,
                                  lens, window, sinks, d ** -0.5 if scale is None else scale,
                                  rows=rows)
    tokens = min(int(max(lens)), window + sinks) if window else int(max(lens))
    weight = None if dtype == "f32" else dtype
    vmax = float(vc.float().abs().max())
    assert_within(out, ref, bound(ref, spread, size, tokens, dtype, weight, vmax))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("heads", [(8, 8), (32, 8), (10, 2), (16, 2)], ids=["g1", "g4", "g5", "g8"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (16, 1), (100, 4), (129, 40)])
def test_decode_matches_oracle(gpu, dtype, head_dim, heads, window, sinks):
    hq, hkv = heads
    q, kc, vc, tables, lens = decode_case(gpu, LENS, hq, hkv, head_dim, dtype, window, sinks,
                                          seed=300 + hq + head_dim + window)
    bt, cl = to_dev(gpu, tables, lens)
    out = pa.paged_attention_decode_window(q, kc, vc, bt, cl, window, sinks, head_dim ** -0.5)
    pa.check_status()
    check_decode(out, q, kc, vc, tables, lens, window, sinks, dtype)
    assert (out[0] == 0).all()


@pytest.mark.parametrize("window,sinks", [(1, 200), (7, 15), (7, 16), (7, 17), (15, 3), (17, 3),
                                          (31, 31), (33, 33), (48, 64), (1998, 1), (1999, 1),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (5, 2 ** 31 - 1)])
def test_decode_window_edges(gpu, window, sinks):
    lens = [1, 5, 16, 17, 31, 32, 33, 47, 48, 49, 64, 65, 80, 97, 1999]
    q, kc, vc, tables, lens = decode_case(gpu, lens, 8, 2, 128, "bf16", window, sinks, seed=41)
    bt, cl = to_dev(gpu, tables, lens)
    out = pa.paged_attention_decode_window(q, kc, vc, bt, cl, window, sinks, 128 ** -0.5)
    pa.check_status()
    check_decode(out, q, kc, vc, tables, lens, window, sinks, "bf16")


def test_window_past_the_context_is_no_window(gpu):
    """Bit for bit: a window of the context's length and more, and none."""
    q, kc, vc, tables, lens = decode_case(gpu, [700, 33, 1], 32, 8, 128, "bf16", 0, 0, seed=43)
    bt, cl = to_dev(gpu, tables, lens)
    outs = [pa.paged_attention_decode_window(q, kc, vc, bt, cl, w, s, 0.1)
            for w, s in ((0, 0), (0, 9), (700, 0), (5000, 3))]
    pa.check_status()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_masked_slots_may_hold_anything(gpu, dtype):
    """NaN and infinities in every slot that nothing sees (blocks behind the
    window that are still in the table, the first tokens' block past them, the
    last block past the context) leave the result bit for bit as it was."""
    window, sinks = 37, 5
    lens = np.array([200, 41, 64, 90, 1], dtype=np.int32)
    gen = np.random.default_rng(47)
    tables, nb = window_tables(lens, lens, 0, 0, gen)      # every block in place
    kc, vc = cache16(nb, 2, 128, dtype, 47, gpu)
    q = wl.normal((5, 8, 128), TORCH_DTYPES[dtype], 471, gpu)
    bt, cl = to_dev(gpu, tables, lens)
    clean = pa.paged_attention_decode_window(q, kc, vc, bt, cl, window, sinks, 0.09)
    keep = torch.zeros((nb, 16), dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in ow.visible_tokens(int(n) - 1, window, sinks):
            keep[int(tables[b, t // 16]), t % 16] = True
    hide = ~keep.to(gpu)[:, None, :, None].expand_as(kc)
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(kc.dtype).min):
        dirty = [c.masked_fill(hide, bad) for c in (kc, vc)]
        out = pa.paged_attention_decode_window(q, *dirty, bt, cl, window, sinks, 0.09)
        assert torch.equal(out, clean)
    pa.check_status()


def test_freed_entries_are_not_read(gpu):
    """Wild table entries for freed blocks set no status; one for a visible
    block does."""
    q, kc, vc, tables, lens = decode_case(gpu, [400, 77], 8, 2, 64, "f16", 40, 3, seed=53)
    tables[tables < 0] = 1 << 30
    bt, cl = to_dev(gpu, tables, lens)
    out = pa.paged_attention_decode_window(q, kc, vc, bt, cl, 40, 3, 0.125)
    pa.check_status()
    tables = np.where(tables == 1 << 30, -1, tables)
    check_decode(out, q, kc, vc, tables, lens, 40, 3, "f16", scale=0.125)
    bt[0, 24] = kc.shape[0]
    pa.paged_attention_decode_window(q, kc, vc, bt, cl, 40, 3, 0.125)
    with pytest.raises(pa.PagedAttnError) as e:
        pa.check_status()
    assert e.value.status == 5


def test_one_plan_many_runs(gpu):
    """One plan in an uninitialised workspace serves runs over several caches;
    repeats are bit-identical, the one-shot call agrees."""
    q, kc, vc, tables, lens = decode_case(gpu, [2000, 5, 0, 900, 16], 32, 8, 128, "bf16", 500, 4, seed=59)
    bt, cl = to_dev(gpu, tables, lens)
    mb = tables.shape[1]
    ws = pa.alloc_window_workspace(5, 32, 8, 128, mb, gpu).fill_(0xA5)
    pa.paged_attention_decode_window_plan(cl, 500, 4, 32, 8, 128, mb, ws)
    one = pa.paged_attention_decode_window(q, kc, vc, bt, cl, 500, 4, 0.1)
    for layer in range(4):
        k2, v2 = (kc, vc) if layer % 2 == 0 else (vc, kc)
        out = pa.paged_attention_decode_window_run(q, k2, v2, bt, cl, 500, 4, 0.1, ws)
        if layer % 2 == 0:
            assert torch.equal(out, one)
    pa.check_status()


def test_a_run_needs_its_plan(gpu):
    q, kc, vc, tables, lens = decode_case(gpu, [100, 20], 8, 2, 64, "f16", 30, 2, seed=61)
    bt, cl = to_dev(gpu, tables, lens)
    mb = tables.shape[1]
    ws = torch.zeros_like(pa.alloc_window_workspace(2, 8, 2, 64, mb, gpu))
    out = torch.full_like(q, 7.0)
    for planned in (None, (31, 2), (30, 3)):
        if planned:
            pa.paged_attention_decode_window_plan(cl, *planned, 8, 2, 64, mb, ws)
        pa.paged_attention_decode_window_run(q, kc, vc, bt, cl, 30, 2, 0.1, ws, out=out)
        with pytest.raises(pa.PagedAttnError) as e:
            pa.check_status()
        assert e.value.status == 1
    assert (out == 7.0).all()


def test_lengths_out_of_range(gpu):
    q, kc, vc, tables, lens = decode_case(gpu, [64, 20], 8, 2, 64, "f16", 16, 0, seed=67)
    bt, cl = to_dev(gpu, tables, lens)
    for bad in (-3, tables.shape[1] * 16 + 1):
        cl[0] = bad
        out = pa.paged_attention_decode_window(q, kc, vc, bt, cl, 16, 0, 0.125)
        with pytest.raises(pa.PagedAttnError) as e:
            pa.check_status()
        assert e.value.status == 5
        assert torch.isfinite(out).all()


def test_other_stream_and_captured_graph(gpu):
    """Plan and run captured once and replayed over changed inputs, on a
    stream of their own."""
    q, kc, vc, tables, lens = decode_case(gpu, [900, 30, 333], 32, 8, 128, "bf16", 256, 4, seed=71)
    bt, cl = to_dev(gpu, tables, lens)
    mb = tables.shape[1]
    ws = pa.alloc_window_workspace(3, 32, 8, 128, mb, gpu)
    out = torch.empty_like(q)
    want = pa.paged_attention_decode_window(q, kc, vc, bt, cl, 256, 4, 0.1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.paged_attention_decode_window_plan(cl, 256, 4, 32, 8, 128, mb, ws)
        pa.paged_attention_decode_window_run(q, kc, vc, bt, cl, 256, 4, 0.1, ws, out=out)
        pa.paged_attention_decode_window_run(q, kc, vc, bt, cl, 256, 4, 0.1, ws, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    cl[1] = 17
    q2 = wl.normal(q.shape, q.dtype, 99, gpu)
    q.copy_(q2)
    graph.replay()
    torch.cuda.synchronize()
    lens[1] = 17
    check_decode(out, q, kc, vc, tables, lens, 256, 4, "bf16", scale=0.1)
    pa.check_status()


def test_blocks_may_sit_anywhere(gpu):
    q, kc, vc, tables, lens = decode_case(gpu, [700, 64, 1], 8, 8, 128, "f16", 300, 20, seed=73)
    bt, cl = to_dev(gpu, tables, lens)
    out = pa.paged_attention_decode_window(q, kc, vc, bt, cl, 300, 20, 0.1)
    perm = np.random.default_rng(1).permutation(kc.shape[0])
    inverse = torch.from_numpy(np.argsort(perm)).to(gpu)
    moved = np.where(tables >= 0, perm[np.maximum(tables, 0)], -1).astype(np.int32)
    out2 = pa.paged_attention_decode_window(q, kc[inverse].contiguous(), vc[inverse].contiguous(),
                                            torch.from_numpy(moved).to(gpu), cl, 300, 20, 0.1)
    pa.check_status()
    assert torch.equal(out, out2)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_many_and_long_sequences(gpu, dtype):
    """Hundreds of short sequences beside a few long ones (sampled against the
    oracle), and one sequence alone."""
    gen = np.random.default_rng(79)
    lens = np.concatenate([gen.integers(0, 60, 700), [20000, 12345, 7777], gen.integers(0, 60, 300)])
    q, kc, vc, tables, lens = decode_case(gpu, lens, 8, 4, 128, dtype, 9000, 33, seed=79)
    bt, cl = to_dev(gpu, tables, lens)
    out = pa.paged_attention_decode_window(q, kc, vc, bt, cl, 9000, 33, 128 ** -0.5)
    pa.check_status()
    rows = {0, 1, 350, 699, 700, 701, 702, 703, 1002}
    check_decode(out, q, kc, vc, tables, lens, 9000, 33, dtype, rows=rows)
    out = pa.paged_attention_decode_window(q[700:701], kc, vc, bt[700:701], cl[700:701], 9000, 33,
                                           128 ** -0.5)
    check_decode(out, q[700:701], kc, vc, tables[700:701], lens[700:701], 9000, 33, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
def test_one_sequence_over_every_sm(gpu, dtype, head_dim):
    """One KV head, one context long enough to be cut into a piece per CTA."""
    q, kc, vc, tables, lens = decode_case(gpu, [70001], 8, 1, head_dim, dtype, 69990, 7, seed=81)
    bt, cl = to_dev(gpu, tables, lens)
    out = pa.paged_attention_decode_window(q, kc, vc, bt, cl, 69990, 7, head_dim ** -0.5)
    pa.check_status()
    check_decode(out, q, kc, vc, tables, lens, 69990, 7, dtype)
    again = pa.paged_attention_decode_window(q, kc, vc, bt, cl, 69990, 7, head_dim ** -0.5)
    assert torch.equal(out, again)


def test_nothing_to_attend(gpu):
    """Every sequence empty: zeros, whatever out held."""
    q, kc, vc, tables, _ = decode_case(gpu, [1, 1, 1], 8, 2, 64, "bf16", 0, 0, seed=87)
    bt, cl = to_dev(gpu, tables, [0, 0, 0])
    out = torch.full_like(q, float("nan"))
    pa.paged_attention_decode_window(q, kc, vc, bt, cl, 3, 1, 0.1, out=out)
    pa.check_status()
    assert (out == 0).all()


@pytest.mark.parametrize("scale", [-0.11, 0.0])
def test_any_sign_of_scale(gpu, scale):
    q, kc, vc, tables, lens = decode_case(gpu, [300, 17], 8, 2, 128, "bf16", 100, 4, seed=91)
    bt, cl = to_dev(gpu, tables, lens)
    out = pa.paged_attention_decode_window(q, kc, vc, bt, cl, 100, 4, scale)
    check_decode(out, q, kc, vc, tables, lens, 100, 4, "bf16", scale=scale)
    st = to_dev(gpu, [0, 1, 2])[0]
    pre = pa.paged_attention_prefill_window(q, kc, vc, bt, cl, st, 100, 4, scale)
    pa.check_status()
    check_decode(pre, q, kc, vc, tables, lens, 100, 4, "bf16", scale=scale)


def test_two_streams_at_once(gpu):
    """Two steps on two streams with a workspace each, interleaved."""
    cases = [decode_case(gpu, lens, 32, 8, 128, "bf16", w, 4, seed=93 + w)
             for lens, w in (([3000, 50, 700], 600), ([90, 2500, 1, 40], 1000))]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    want, got, keep = [], [[], []], []
    for (q, kc, vc, tables, lens), w in zip(cases, (600, 1000)):
        bt, cl = to_dev(gpu, tables, lens)
        ws = pa.alloc_window_workspace(len(lens), 32, 8, 128, tables.shape[1], gpu)
        keep.append((bt, cl, ws))
        want.append(pa.paged_attention_decode_window(q, kc, vc, bt, cl, w, 4, 0.1))
    torch.cuda.synchronize()
    for _ in range(20):
        for i, ((q, kc, vc, tables, lens), w) in enumerate(zip(cases, (600, 1000))):
            with torch.cuda.stream(streams[i]):
                bt, cl, ws = keep[i]
                got[i].append(pa.paged_attention_decode_window(q, kc, vc, bt, cl, w, 4, 0.1, workspace=ws))
    torch.cuda.synchronize()
    pa.check_status()
    for i in range(2):
        for out in got[i]:
            assert torch.equal(out, want[i])


def test_cache_past_32_bit_offsets(gpu):
    """A cache of more than 2^32 elements, the visible blocks at its end."""
    nb = (1 << 32) // (8 * 16 * 128) + 64
    kc = torch.zeros((nb, 8, 16, 128), dtype=torch.bfloat16, device=gpu)
    vc = torch.zeros_like(kc)
    small = cache16(40, 8, 128, "bf16", 83, gpu)
    kc[-40:], vc[-40:] = small[0], small[1]
    tables = (nb - 1 - np.arange(40)[None]).astype(np.int32)
    bt, cl = to_dev(gpu, tables, [635])
    q = wl.normal((1, 32, 128), torch.bfloat16, 831, gpu)
    out = pa.paged_attention_decode_window(q, kc, vc, bt, cl, 300, 4, 0.1)
    low = pa.paged_attention_decode_window(q, *small, bt - (nb - 40), cl, 300, 4, 0.1)
    pa.check_status()
    assert torch.equal(out, low)


# ------------------------------------------------------------------ prefill
PLENS = [40, 17, 300, 1, 530, 1500, 64, 900, 16]
PNEW = [40, 17, 37, 1, 1, 9, 0, 128, 16]


def prefill_case(dev, lens, new, hq, hkv, d, dtype, window, sinks, seed):
    gen = np.random.default_rng(seed)
    tables, nb = window_tables(lens, new, window, sinks, gen)
    kc, vc = cache16(nb, hkv, d, dtype, seed, dev)
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = wl.normal((int(qs[-1]), hq, d), TORCH_DTYPES[dtype], seed * 10 + 1, dev)
    return q, kc, vc, tables, np.asarray(lens, dtype=np.int32), qs


def check_prefill(out, q, kc, vc, tables, lens, qs, window, sinks, dtype, rows=None):
    d = q.shape[2]
    ref, spread, size = ow.prefill(to_f32_numpy(q), to_f32_numpy(kc), to_f32_numpy(vc), tables,
                                   lens, qs, window, sinks, d ** -0.5, rows=rows)
    tokens = min(int(max(lens)), window + sinks) if window else int(max(lens))
    weight = None if dtype == "f32" else dtype
    vmax = float(vc.float().abs().max())
    assert_within(out, ref, bound(ref, spread, size, tokens, dtype, weight, vmax))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("heads", [(4, 4), (8, 2), (5, 1), (8, 1)], ids=["g1", "g4", "g5", "g8"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 1), (100, 4), (129, 40), (4000, 4)])
def test_prefill_matches_oracle(gpu, dtype, head_dim, heads, window, sinks):
    hq, hkv = heads
    q, kc, vc, tables, lens, qs = prefill_case(gpu, PLENS, PNEW, hq, hkv, head_dim, dtype, window,
                                               sinks, seed=500 + hq + head_dim + window)
    bt, cl, st = to_dev(gpu, tables, lens, qs)
    out = pa.paged_attention_prefill_window(q, kc, vc, bt, cl, st, window, sinks, head_dim ** -0.5)
    pa.check_status()
    rows = set(range(0, 60)) | set(range(60, int(qs[-1]), 7))
    check_prefill(out, q, kc, vc, tables, lens, qs, window, sinks, dtype, rows)


@pytest.mark.parametrize("window,sinks", [(1, 300), (7, 15), (7, 16), (15, 3), (17, 17), (48, 64),
                                          (127, 4), (128, 128), (129, 0), (256, 5), (257, 129),
                                          (640, 1), (2 ** 31 - 1, 2 ** 31 - 1), (5, 2 ** 31 - 1)])
@pytest.mark.parametrize("head_dim", [64, 128])
def test_prefill_window_edges(gpu, window, sinks, head_dim):
    """Chunks that begin inside, at and past the window; the first tokens'
    blocks next to, inside and away from it."""
    lens, new = [700, 129, 641, 128, 300], [300, 129, 2, 64, 41]
    q, kc, vc, tables, lens, qs = prefill_case(gpu, lens, new, 4, 1, head_dim, "bf16", window,
                                               sinks, seed=61)
    bt, cl, st = to_dev(gpu, tables, lens, qs)
    out = pa.paged_attention_prefill_window(q, kc, vc, bt, cl, st, window, sinks, head_dim ** -0.5)
    pa.check_status()
    check_prefill(out, q, kc, vc, tables, lens, qs, window, sinks, "bf16",
                  set(range(0, int(qs[-1]), 5)))


def test_prefill_without_a_window_is_prefill(gpu):
    q, kc, vc, tables, lens, qs = prefill_case(gpu, PLENS, PNEW, 8, 2, 128, "bf16", 0, 0, seed=67)
    bt, cl, st = to_dev(gpu, tables, lens, qs)
    a, b = torch.full_like(q, 3.0), torch.full_like(q, 3.0)
    pa.paged_attention_prefill(q, kc, vc, bt, cl, st, 0.1, out=a)
    pa.paged_attention_prefill_window(q, kc, vc, bt, cl, st, 0, 5, 0.1, out=b)
    pa.check_status()
    assert torch.equal(a, b)


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_prefill_masked_slots_may_hold_anything(gpu, dtype, head_dim):
    """Slots that no row of a chunk sees hold NaN or infinities: nothing
    changes, bit for bit."""
    window, sinks = 70, 5
    lens, new = np.array([500, 130, 90]), np.array([150, 40, 90])
    gen = np.random.default_rng(71)
    tables, nb = window_tables(lens, lens, 0, 0, gen)
    kc, vc = cache16(nb, 2, head_dim, dtype, 71, gpu)
    qs = np.concatenate([[0], np.cumsum(new)])
    q = wl.normal((int(qs[-1]), 8, head_dim), TORCH_DTYPES[dtype], 711, gpu)
    bt, cl, st = to_dev(gpu, tables, lens, qs)
    clean = pa.paged_attention_prefill_window(q, kc, vc, bt, cl, st, window, sinks, 0.09)
    keep = torch.zeros((nb, 16), dtype=torch.bool)
    for b in range(3):
        for p in range(lens[b] - new[b], lens[b]):
            for t in ow.visible_tokens(int(p), window, sinks):
                keep[int(tables[b, t // 16]), t % 16] = True
    hide = ~keep.to(gpu)[:, None, :, None].expand_as(kc)
    for bad in (float("nan"), float("inf"), torch.finfo(kc.dtype).min):
        dirty = [c.masked_fill(hide, bad) for c in (kc, vc)]
        out = pa.paged_attention_prefill_window(q, *dirty, bt, cl, st, window, sinks, 0.09)
        assert torch.equal(out, clean)
    pa.check_status()


def test_prefill_plan_and_rows_of_no_sequence(gpu):
    """One plan, several runs; rows behind the last sequence and of an idle
    one are left as they were; a run without its plan does nothing."""
    q, kc, vc, tables, lens, qs = prefill_case(gpu, PLENS, PNEW, 8, 2, 128, "bf16", 90, 4, seed=73)
    total = int(qs[-1]) + 11
    q = torch.cat([q, torch.full((11, 8, 128), float("nan"), dtype=q.dtype, device=gpu)])
    bt, cl, st = to_dev(gpu, tables, lens, qs)
    mb = tables.shape[1]
    ws = pa.alloc_prefill_workspace(len(lens), total, 8, 2, 128, gpu).fill_(0xA5)
    pa.paged_attention_prefill_window_plan(cl, st, total, 90, 4, 8, 2, 128, mb, 0.1,
                                           torch.bfloat16, ws)
    outs = []
    for _ in range(3):
        out = torch.full_like(q, 5.0)
        pa.paged_attention_prefill_window_run(q, kc, vc, bt, cl, st, 90, 4, 0.1, ws, out=out)
        outs.append(out)
    pa.check_status()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert (outs[0][-11:] == 5.0).all() and torch.isfinite(outs[0][:-11]).all()
    pa.paged_attention_prefill_window_run(q, kc, vc, bt, cl, st, 91, 4, 0.1, ws, out=outs[1])
    with pytest.raises(pa.PagedAttnError) as e:
        pa.check_status()
    assert e.value.status == 1
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("lens,new", [([9000, 12345], [3, 16]), ([5000], [700]),
                                      ([2048, 4096, 6000], [2048, 1000, 77])])
def test_prefill_long_contexts(gpu, lens, new):
    """Long windows over few and many rows (split key ranges among them)."""
    q, kc, vc, tables, lens, qs = prefill_case(gpu, lens, new, 8, 2, 128, "bf16", 3000, 200, seed=79)
    bt, cl, st = to_dev(gpu, tables, lens, qs)
    out = pa.paged_attention_prefill_window(q, kc, vc, bt, cl, st, 3000, 200, 128 ** -0.5)
    pa.check_status()
    rows = set(np.linspace(0, int(qs[-1]) - 1, 9).astype(int).tolist())
    check_prefill(out, q, kc, vc, tables, lens, qs, 3000, 200, "bf16", rows)
    again = pa.paged_attention_prefill_window(q, kc, vc, bt, cl, st, 3000, 200, 128 ** -0.5)
    assert torch.equal(out, again)


@pytest.mark.parametrize("window,sinks", [(100, 4), (600, 30)])
@pytest.mark.parametrize("heads", [(8, 8), (8, 2)], ids=["g1", "g4"])
def test_prefill_rows_rescale_apart(gpu, heads, window, sinks):
    """Keys grow along the sequence and few rows have large queries: within a
    warp some rows' softmax references move, others' do not, and rows whose
    window begins later have seen nothing yet."""
    hq, hkv = heads
    lens, new = [900, 1500, 130], [260, 700, 130]
    gen = np.random.default_rng(5)
    tables, nb = window_tables(lens, new, window, sinks, gen)
    grow = np.ones(nb, dtype=np.float32)
    for b, n in enumerate(lens):
        for j in range((n + 15) // 16):
            if tables[b, j] >= 0:
                grow[tables[b, j]] = 2.0 ** min(3.0, j / 12)
    shape = (nb, hkv, 16, 128)
    kc = (wl.normal(shape, torch.float32, 213, gpu) * torch.from_numpy(grow).to(gpu)[:, None, None, None]).bfloat16()
    vc = wl.normal(shape, torch.bfloat16, 214, gpu)
    qs = np.concatenate([[0], np.cumsum(new)])
    size = np.where(gen.random((int(qs[-1]), hq, 1)) < 0.1, 4.0, 0.25).astype(np.float32)
    q = (wl.normal((int(qs[-1]), hq, 128), torch.float32, 215, gpu) * torch.from_numpy(size).to(gpu)).bfloat16()
    lens = np.asarray(lens)
    bt, cl, st = to_dev(gpu, tables, lens, qs)
    out = pa.paged_attention_prefill_window(q, kc, vc, bt, cl, st, window, sinks, 128 ** -0.5)
    pa.check_status()
    check_prefill(out, q, kc, vc, tables, lens, qs, window, sinks, "bf16", set(range(0, int(qs[-1]), 13)))
    again = pa.paged_attention_prefill_window(q, kc, vc, bt, cl, st, window, sinks, 128 ** -0.5)
    assert torch.equal(out, again)
