"""Append and decode of an 8-bit cache in one launch: bit for bit what the two
calls give, and codes and scales the oracle's."""

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from oracle import cache_q8 as oq
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.gpu_helpers import TORCH_DTYPES, to_f32_numpy
from tests.test_gpu_q8 import Mirror, check_decode, codes_of
from tests.test_gpu_window import to_dev
from tests.window_helpers import window_tables

pytestmark = pytest.mark.gpu

# no token, one, a block's first and last slot, many blocks; the odd ones in front of, between and
# behind the others
LENS = [0, 1, 2, 15, 16, 17, 32, 0, 33, 100, 257, 530, 1999, 0]


def copies(m):
    return [[c.clone() for c in m.dcodes], [s.clone() for s in m.dscales]]


def both(q, k, v, m, tables, lens, window, sinks, scale, dev):
    """The cache after and the output of one launch (on m) and of the two calls."""
    codes, scales = copies(m)
    bt, cl, st = to_dev(dev, tables, lens, range(len(lens) + 1))
    hq, hkv, d = q.shape[1], k.shape[1], q.shape[2]
    ws = pa.alloc_window_workspace(len(lens), hq, hkv, d, tables.shape[1], dev)
    pa.paged_attention_decode_window_plan(cl, window, sinks, hq, hkv, d, tables.shape[1], ws)
    one = pa.paged_attention_decode_q8_append_run(q, k, v, *m.dcodes, *m.dscales, bt, cl, window, sinks,
                                                  scale, ws)
    # (the append takes no token for a sequence without tokens)
    has = [b for b, n in enumerate(lens) if n > 0]
    keep = torch.tensor(has, dtype=torch.long, device=dev)
    starts = torch.from_numpy(np.concatenate([[0], np.cumsum(np.asarray(lens) > 0)]).astype(np.int32)).to(dev)
    pa.kv_append_q8(k[keep].contiguous(), v[keep].contiguous(), *codes, *scales, bt, cl, starts)
    two = pa.paged_attention_decode_q8_run(q, *codes, *scales, bt, cl, window, sinks, scale, ws)
    return one, two, codes, scales


def check_same(m, one, two, codes, scales):
    for i in range(2):
        np.testing.assert_array_equal(codes_of(m.dcodes[i]), codes_of(codes[i]))
        assert torch.equal(m.dscales[i].view(torch.int32), scales[i].view(torch.int32))
    assert torch.equal(one.view(torch.int16), two.view(torch.int16))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("heads", [(8, 8), (32, 8), (10, 2), (8, 1)], ids=["g1", "g4", "g5", "g8"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 4)])
def test_matches_both_calls_and_oracle(gpu, dtype, head_dim, heads, window, sinks):
    hq, hkv = heads
    gen = np.random.default_rng(hq + window + head_dim)
    tables, nb = window_tables(LENS, [1] * len(LENS), window, sinks, gen)
    n = len(LENS)
    # the new rows from far under to far over what the blocks hold: scales that stay and that grow
    for size in (0.05, 1.0, 40.0):
        m = Mirror(nb, hkv, head_dim, 29 + hq, gpu)
        q = wl.normal((n, hq, head_dim), TORCH_DTYPES[dtype], 31 + window, gpu)
        k, v = (wl.normal((n, hkv, head_dim), TORCH_DTYPES[dtype], 51 + i, gpu) * size for i in range(2))
        one, two, codes, scales = both(q, k, v, m, tables, LENS, window, sinks, head_dim ** -0.5, gpu)
        pa.check_status()
        check_same(m, one, two, codes, scales)
        has = np.asarray(LENS) > 0
        oq.kv_append_q8(to_f32_numpy(k)[has], to_f32_numpy(v)[has], *m.codes, *m.scales, tables, LENS,
                        np.concatenate([[0], np.cumsum(has)]))
        m.check()
        check_decode(one, q, m, tables, LENS, window, sinks, dtype)
        assert (one[~torch.from_numpy(has)] == 0).all()


def test_values_without_a_scale(gpu):
    """Zeros, infinities and NaN among the new rows, K and V apart."""
    lens = [1, 1, 17, 18, 40, 31]
    gen = np.random.default_rng(3)
    tables, nb = window_tables(lens, [1] * 6, 0, 0, gen)
    q = wl.normal((6, 8, 64), torch.bfloat16, 5, gpu)
    k, v = (wl.normal((6, 2, 64), torch.bfloat16, 7 + i, gpu) for i in range(2))
    k[0], v[1], k[2, 0, 3], v[3, 1, 60] = 0, 0, float("inf"), float("nan")
    k[4], v[5] = float("nan"), -float("inf")
    m = Mirror(nb, 2, 64, 9, gpu)
    one, two, codes, scales = both(q, k, v, m, tables, lens, 0, 0, 0.125, gpu)
    pa.check_status()
    for i in range(2):
        np.testing.assert_array_equal(codes_of(m.dcodes[i]), codes_of(codes[i]))
        assert torch.equal(m.dscales[i], scales[i])
    same = (one == two) | (one.isnan() & two.isnan())
    assert same.all()


def test_batches_of_every_size(gpu):
    """One short sequence, a batch of single tokens, one that fills every SM:
    shares from one block to many, a warp's blocks over several sequences."""
    gen = np.random.default_rng(11)
    for lens in ([5], [1] * 300, [40000], list(gen.integers(0, 90, 513)), [3, 30000, 4]):
        tables, nb = window_tables(lens, [1] * len(lens), 0, 0, gen)
        m = Mirror(nb, 4, 128, 13, gpu)
        q = wl.normal((len(lens), 16, 128), torch.bfloat16, 15, gpu)
        k, v = (wl.normal((len(lens), 4, 128), torch.bfloat16, 17 + i, gpu) * 2 for i in range(2))
        one, two, codes, scales = both(q, k, v, m, tables, lens, 0, 0, 128 ** -0.5, gpu)
        pa.check_status()
        check_same(m, one, two, codes, scales)


@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_bad_block_stores_nothing(gpu, bad):
    lens = [20, 33, 48]
    gen = np.random.default_rng(19)
    tables, nb = window_tables(lens, [1] * 3, 0, 0, gen)
    q = wl.normal((3, 8, 128), torch.bfloat16, 21, gpu)
    k, v = (wl.normal((3, 2, 128), torch.bfloat16, 23 + i, gpu) * 30 for i in range(2))
    m = Mirror(nb, 2, 128, 25, gpu)
    dirty = tables.copy()
    dirty[1, 2] = bad
    bt, cl = to_dev(gpu, dirty, lens)
    ws = pa.alloc_window_workspace(3, 8, 2, 128, 3, gpu)
    pa.paged_attention_decode_window_plan(cl, 0, 0, 8, 2, 128, 3, ws)
    out = pa.paged_attention_decode_q8_append_run(q, k, v, *m.dcodes, *m.dscales, bt, cl, 0, 0, 0.1, ws)
    with pytest.raises(pa.PagedAttnError) as e:
        pa.check_status()
    assert e.value.status == 5
    for b in (0, 2):
        oq.kv_append_q8(to_f32_numpy(k)[b:b + 1], to_f32_numpy(v)[b:b + 1], *m.codes, *m.scales,
                        tables[b:b + 1], lens[b:b + 1], [0, 1])
    m.check()
    check_decode(out, q, m, tables, lens, 0, 0, "bf16", rows={0, 2}, scale=0.1)


@pytest.mark.parametrize("now,status", [([20, 34, 48], 1), ([20, 32, 48], 1), ([20, 0, 48], 1),
                                        ([20, -5, 48], 1), ([20, 49, 48], 5)])
def test_other_length_stores_nothing(gpu, now, status):
    """A length that is not the planned one, or that the table cannot hold
    (planned as it is): nothing is stored for that sequence, its query sees the
    cache as it was."""
    lens = [20, 33, 48] if status == 1 else now
    gen = np.random.default_rng(35)
    tables, nb = window_tables([20, 33, 48], [1] * 3, 0, 0, gen)
    if status == 5:
        tables, nb = window_tables([20, 48, 48], [1] * 3, 0, 0, gen)
    q = wl.normal((3, 8, 64), torch.float16, 37, gpu)
    k, v = (wl.normal((3, 2, 64), torch.float16, 39 + i, gpu) * 30 for i in range(2))
    m = Mirror(nb, 2, 64, 41, gpu)
    bt, cl = to_dev(gpu, tables, lens)
    ws = pa.alloc_window_workspace(3, 8, 2, 64, 3, gpu)
    pa.paged_attention_decode_window_plan(cl, 0, 0, 8, 2, 64, 3, ws)
    cl.copy_(torch.tensor(now, dtype=torch.int32))
    out = pa.paged_attention_decode_q8_append_run(q, k, v, *m.dcodes, *m.dscales, bt, cl, 0, 0, 0.1, ws)
    with pytest.raises(pa.PagedAttnError) as e:
        pa.check_status()
    assert e.value.status == status
    for b in (0, 2):
        oq.kv_append_q8(to_f32_numpy(k)[b:b + 1], to_f32_numpy(v)[b:b + 1], *m.codes, *m.scales,
                        tables[b:b + 1], now[b:b + 1], [0, 1])
    m.check()
    seen = [min(n, 48) for n in lens]
    check_decode(out, q, m, tables, seen, 0, 0, "f16", scale=0.1)


def test_captured_layers(gpu):
    """Several layers on one plan, captured and replayed while the sequences
    grow past blocks' ends: each step's cache and output the oracle's."""
    hq, hkv, d, window, sinks, layers = 32, 8, 128, 64, 4, 3
    gen = np.random.default_rng(27)
    lens = np.array([90, 16, 31, 200])
    tables, nb = window_tables(lens + 20, lens + 20, 0, 0, gen)
    mirrors = [Mirror(nb, hkv, d, 29 + i, gpu) for i in range(layers)]
    bt, cl = to_dev(gpu, tables, lens)
    k, v = (torch.zeros((4, hkv, d), dtype=torch.bfloat16, device=gpu) for _ in range(2))
    q = torch.zeros((4, hq, d), dtype=torch.bfloat16, device=gpu)
    outs = [torch.zeros_like(q) for _ in range(layers)]
    ws = pa.alloc_window_workspace(4, hq, hkv, d, tables.shape[1], gpu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.paged_attention_decode_window_plan(cl, window, sinks, hq, hkv, d, tables.shape[1], ws)
        ops = [pa.prepare_decode_q8_append_run(q, k, v, *m.dcodes, *m.dscales, bt, cl, window, sinks,
                                               d ** -0.5, ws, out) for m, out in zip(mirrors, outs)]
        for op in ops:
            op()
    for step in range(1, 20):
        lens = lens + 1
        cl += 1
        for i, t in enumerate((k, v, q)):
            t.copy_(wl.normal(tuple(t.shape), t.dtype, 1000 * step + i, gpu) * (1 + step % 3))
        graph.replay()
        torch.cuda.synchronize()
        for m, out in zip(mirrors, outs):
            oq.kv_append_q8(to_f32_numpy(k), to_f32_numpy(v), *m.codes, *m.scales, tables, lens, range(5))
            m.check()
            check_decode(out, q, m, tables, lens, window, sinks, "bf16")
    pa.check_status()


def test_python_refusals(gpu):
    m = Mirror(4, 2, 64, 33, gpu)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device=gpu)
    k = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device=gpu)
    bt, cl = to_dev(gpu, np.zeros((1, 1), dtype=np.int32), [1])
    ws = pa.alloc_window_workspace(1, 4, 2, 64, 1, gpu)
    for kn, vn in ((k.half(), k.half()), (k[:, :1].contiguous(), k), (k, k[..., :32].contiguous()),
                   (k, k.cpu()), (k.expand(2, 2, 64)[:, :1], k)):
        with pytest.raises((ValueError, TypeError, pa.PagedAttnError)):
            pa.paged_attention_decode_q8_append_run(q, kn, vn, *m.dcodes, *m.dscales, bt, cl, 0, 0, 0.1, ws)
