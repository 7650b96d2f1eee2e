"""Rotation on the way into the caches: bit for bit the rotation followed by
the append that is there, and everything else left as it was."""

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.gpu_helpers import TORCH_DTYPES
from tests.rotary_helpers import bits, projection, rotary_of, same_bits
from tests.test_gpu_q8 import ALENS, ANEW
from tests.test_gpu_window import to_dev
from tests.window_helpers import cache8, cache16, window_tables

pytestmark = pytest.mark.gpu


def slots_of(n, nb, gen):
    return torch.from_numpy(gen.permutation(nb * 16)[:n].astype(np.int64))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("heads", [(32, 8), (3, 3), (10, 2), (64, 64)], ids=str)
@pytest.mark.parametrize("n", [1, 97])
def test_append_is_rotary_then_append(gpu, dtype, head_dim, heads, n):
    hq, hkv = heads
    rot, _ = rotary_of(pa, head_dim, gpu, head_dim // 2 if n > 1 else None, hkv == 3, 1.1)
    q, k, v = projection(n, hq, hkv, head_dim, dtype, 3 + hq, gpu, pad=8)
    nb = 12
    gen = np.random.default_rng(hq + n)
    slots = slots_of(n, nb, gen)
    slots[::5] = -1                                     # padding
    slots = slots.to(gpu)
    pos = torch.from_numpy(gen.integers(0, 100000, n).astype(np.int32)).to(gpu)
    kc, vc = cache16(nb, hkv, head_dim, dtype, 7, gpu)
    kw, vw = kc.clone(), vc.clone()
    qo, ko = pa.rotary(q, k, pos, rot)
    pa.kv_append(ko, v.contiguous(), kw, vw, slots)
    got = pa.rotary_kv_append(q, k, v, pos, rot, kc, vc, slots)
    pa.check_status()
    assert same_bits(got, qo) and same_bits(kc, kw) and same_bits(vc, vw)
    # keys alone, and the queries in place
    kc2, vc2 = cache16(nb, hkv, head_dim, dtype, 7, gpu)
    assert pa.rotary_kv_append(None, k, v, pos, rot, kc2, vc2, slots) is None
    assert same_bits(kc2, kw) and same_bits(vc2, vw)
    op = pa.prepare_rotary_kv_append(q, k, v, pos, rot, kc2, vc2, slots, q)
    op()
    assert same_bits(q, qo) and same_bits(kc2, kw)


def test_append_bad_slots(gpu):
    """A slot past the cache stores nothing and is reported; the query is
    rotated all the same."""
    rot, _ = rotary_of(pa, 128, gpu)
    q, k, v = projection(6, 8, 2, 128, "bf16", 3, gpu)
    kc, vc = cache16(4, 2, 128, "bf16", 7, gpu)
    kw, vw = kc.clone(), vc.clone()
    pos = torch.arange(6, dtype=torch.int32, device=gpu)
    slots = torch.tensor([3, 64, 17, 1 << 40, -5, 63], dtype=torch.int64, device=gpu)
    got = pa.rotary_kv_append(q, k, v, pos, rot, kc, vc, slots)
    with pytest.raises(pa.PagedAttnError) as e:
        pa.check_status()
    assert e.value.status == 5
    qo, ko = pa.rotary(q, k, pos, rot)
    keep = torch.tensor([0, 2, 5], device=gpu)
    pa.kv_append(ko[keep], v[keep].contiguous(), kw, vw, slots[keep])
    assert same_bits(got, qo) and same_bits(kc, kw) and same_bits(vc, vw)


def test_append_past_32_bit_offsets(gpu):
    rot, _ = rotary_of(pa, 128, gpu)
    nb = (1 << 31) // (16 * 128) + 100                  # one KV head: elements past 2^31
    kc = torch.zeros((nb, 1, 16, 128), dtype=torch.bfloat16, device=gpu)
    vc = torch.zeros_like(kc)
    q, k, v = projection(3, 1, 1, 128, "bf16", 3, gpu)
    pos = torch.arange(3, dtype=torch.int32, device=gpu)
    slots = torch.tensor([nb * 16 - 1, 5, nb * 16 - 40], dtype=torch.int64, device=gpu)
    qo, ko = pa.rotary(q, k, pos, rot)
    assert same_bits(pa.rotary_kv_append(q, k, v, pos, rot, kc, vc, slots), qo)
    pa.check_status()
    for cache, rows in ((kc, ko), (vc, v)):
        for i, s in enumerate(slots.tolist()):
            assert same_bits(cache[s // 16, 0, s % 16], rows[i, 0])
            cache[s // 16, 0, s % 16] = 0
        assert int(torch.count_nonzero(cache[-8:])) == 0 and int(torch.count_nonzero(cache[:8])) == 0


def q8_case(dev, hkv, d, seed, lens=ALENS, new=ANEW):
    gen = np.random.default_rng(seed)
    qs = np.concatenate([[0], np.cumsum(new)])
    tables, nb = window_tables(lens, lens, 0, 0, gen)
    _, _, codes, scales = cache8(nb, hkv, d, seed, dev)
    return qs, tables, nb, codes, scales


def places(lens, new):
    return np.concatenate([np.arange(c - n, c) for c, n in zip(lens, new)]).astype(np.int32)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("heads", [(32, 8), (5, 5), (7, 1)], ids=str)
@pytest.mark.parametrize("given", [False, True])
def test_append_q8_is_rotary_then_append(gpu, dtype, head_dim, heads, given):
    """Keys rotated in 32 bits and quantised from there; rows behind the last
    sequence left as they were; chunks that begin and end anywhere in a block,
    growing scales among them."""
    hq, hkv = heads
    rot, _ = rotary_of(pa, head_dim, gpu, head_dim // 2 if given else None, given, 0.9)
    qs, tables, nb, codes, scales = q8_case(gpu, hkv, head_dim, 5 + hq)
    total, more = int(qs[-1]), 5
    bt, cl, st = to_dev(gpu, tables, ALENS, qs)
    gen = np.random.default_rng(3)
    where = gen.integers(0, 50000, total + more).astype(np.int32) if given else places(ALENS, ANEW)
    pos = torch.from_numpy(where).to(gpu)
    for step in range(2):
        q, k, v = projection(total + more, hq, hkv, head_dim, dtype, 11 + step, gpu, pad=8)
        k *= torch.exp(2 * torch.randn((total + more, 1, 1), device=gpu)).to(k.dtype)
        want_codes, want_scales = [c.clone() for c in codes], [s.clone() for s in scales]
        wide, _ = pa.rotary(k[:total].float(), None, pos[:total], rot)
        pa.kv_append_q8(wide, v[:total].float().contiguous(), *want_codes, *want_scales, bt, cl, st)
        qo = torch.full((total + more, hq, head_dim), 7.0, dtype=q.dtype, device=gpu)
        got = pa.rotary_kv_append_q8(q, k, v, pos if given else None, rot, *codes, *scales, bt, cl, st, q_out=qo)
        pa.check_status()
        assert got is qo
        assert same_bits(qo[:total], pa.rotary(q[:total], None, pos[:total], rot)[0])
        assert (qo[total:] == 7).all()
        for i in range(2):
            assert same_bits(codes[i], want_codes[i]) and same_bits(scales[i], want_scales[i])


# a decode step; a chunk or two among sequences that have nothing new
FEW = {"step": ([1, 16, 17, 100, 33, 700, 48, 31, 2, 15], [1] * 10),
       "chunks": ([40, 16, 17, 7, 33, 18, 48, 31, 2, 15, 12, 11, 99, 20, 10], [24, 0, 0, 1, 0, 2, 0, 0, 0, 0, 0, 0, 0, 2, 0]),
       "empty": ([5, 0, 9], [0, 0, 1])}


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("heads", [(32, 8), (7, 1), (70, 70)], ids=str)
@pytest.mark.parametrize("shape", sorted(FEW))
def test_append_q8_of_few_tokens(gpu, dtype, head_dim, heads, shape):
    hq, hkv = heads
    lens, new = FEW[shape]
    rot, _ = rotary_of(pa, head_dim, gpu, head_dim // 2, hq == 7, 0.9)
    qs, tables, nb, codes, scales = q8_case(gpu, hkv, head_dim, 5 + hq, lens, new)
    total = int(qs[-1])
    assert total <= 2 * len(lens)
    bt, cl, st = to_dev(gpu, tables, lens, qs)
    pos = torch.from_numpy(places(lens, new)).to(gpu)
    for size in (0.1, 1.0, 30.0):
        q, k, v = projection(total + 2, hq, hkv, head_dim, dtype, 11, gpu, pad=8)
        k *= size
        v *= size
        want = [t.clone() for t in (*codes, *scales)]
        wide, _ = pa.rotary(k[:total].float(), None, pos, rot)
        pa.kv_append_q8(wide, v[:total].float().contiguous(), *want, bt, cl, st)
        qo = torch.full((total + 2, hq, head_dim), 7.0, dtype=q.dtype, device=gpu)
        pa.rotary_kv_append_q8(q, k, v, None, rot, *codes, *scales, bt, cl, st, q_out=qo)
        pa.check_status()
        assert same_bits(qo[:total], pa.rotary(q[:total], None, pos, rot)[0]) and (qo[total:] == 7).all()
        for a, b in zip((*codes, *scales), want):
            assert same_bits(a, b)


def test_append_q8_of_few_tokens_reports(gpu):
    """A bad block, a sequence that runs backwards, one behind it among an
    earlier one's rows, one longer than its table."""
    rot, _ = rotary_of(pa, 64, gpu)
    gen = np.random.default_rng(1)
    lens = [20, 10, 18, 9, 200, 3, 3]
    starts = np.array([0, 4, 1, 6, 7, 8, 8, 8], dtype=np.int32)
    tables, nb = window_tables(np.minimum(lens, 32), np.minimum(lens, 32), 0, 0, gen)
    _, _, codes, scales = cache8(nb, 2, 64, 3, gpu)
    tables[3, 0] = 1 << 20
    q, k, v = projection(8, 4, 2, 64, "bf16", 3, gpu)
    pos = torch.from_numpy(gen.integers(0, 999, 8).astype(np.int32)).to(gpu)
    bt, cl, st = to_dev(gpu, tables, lens, starts)
    want = [t.clone() for t in (*codes, *scales)]
    wide, _ = pa.rotary(k.float(), None, pos, rot)
    pa.kv_append_q8(wide, v.float().contiguous(), *want, bt, cl, st)
    qo = torch.full((8, 4, 64), 7.0, dtype=q.dtype, device=gpu)
    with pytest.raises(pa.PagedAttnError):
        pa.check_status()
    pa.rotary_kv_append_q8(q, k, v, pos, rot, *codes, *scales, bt, cl, st, q_out=qo)
    with pytest.raises(pa.PagedAttnError) as e:
        pa.check_status()
    assert e.value.status == 5
    for a, b in zip((*codes, *scales), want):
        assert same_bits(a, b)
    right = pa.rotary(q, None, pos, rot)[0]
    assert same_bits(qo[:7], right[:7]) and (qo[7:] == 7).all()


def test_append_q8_keys_alone_and_prepared(gpu):
    rot, _ = rotary_of(pa, 128, gpu)
    qs, tables, nb, codes, scales = q8_case(gpu, 2, 128, 5)
    start = [t.clone() for t in (*codes, *scales)]
    total = int(qs[-1])
    bt, cl, st = to_dev(gpu, tables, ALENS, qs)
    q, k, v = projection(total, 8, 2, 128, "bf16", 3, gpu)
    assert pa.rotary_kv_append_q8(None, k, v, None, rot, *codes, *scales, bt, cl, st) is None
    want_q = pa.rotary(q, None, torch.from_numpy(places(ALENS, ANEW)).to(gpu), rot)[0]
    pa.prepare_rotary_kv_append_q8(q, k, v, None, rot, *start, bt, cl, st, q)()
    assert same_bits(q, want_q)
    for a, b in zip((*codes, *scales), start):
        assert same_bits(a, b)
    pa.check_status()


def test_append_q8_special_values(gpu):
    """Zeros, infinities and NaN among the rows."""
    rot, _ = rotary_of(pa, 64, gpu)
    lens = new = [16, 16, 16, 16]
    qs, tables, nb, codes, scales = q8_case(gpu, 2, 64, 9, lens, new)
    bt, cl, st = to_dev(gpu, tables, lens, qs)
    q, k, v = projection(64, 4, 2, 64, "bf16", 3, gpu)
    k[:16], v[:16] = 0, 0
    k[20, 0, 3], v[20, 1, 3] = float("inf"), float("-inf")
    k[40, 1, 40], v[41, 0, 2] = float("nan"), float("nan")
    k[48:] = float("nan")
    want_codes, want_scales = [c.clone() for c in codes], [s.clone() for s in scales]
    pos = torch.from_numpy(places(lens, new)).to(gpu)
    wide, _ = pa.rotary(k.float(), None, pos, rot)
    pa.kv_append_q8(wide, v.float().contiguous(), *want_codes, *want_scales, bt, cl, st)
    pa.rotary_kv_append_q8(q, k, v, None, rot, *codes, *scales, bt, cl, st)
    pa.check_status()
    for i in range(2):
        nan = (bits(want_codes[i]) & 0x7F) == 0x7F
        assert torch.equal(nan, (bits(codes[i]) & 0x7F) == 0x7F)
        assert torch.equal(bits(codes[i])[~nan], bits(want_codes[i])[~nan])
        assert same_bits(scales[i], want_scales[i])


@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_append_q8_bad_block(gpu, bad):
    """A bad block loses its own keys and values; queries are rotated."""
    rot, _ = rotary_of(pa, 128, gpu)
    lens, new = [40, 33], [40, 33]
    qs, tables, nb, codes, scales = q8_case(gpu, 2, 128, 7, lens, new)
    q, k, v = projection(73, 4, 2, 128, "bf16", 3, gpu)
    pos = torch.from_numpy(places(lens, new)).to(gpu)
    dirty = tables.copy()
    dirty[0, 1] = bad
    bt, cl, st = to_dev(gpu, dirty, lens, qs)
    want = [t.clone() for t in (*codes, *scales)]
    clean = to_dev(gpu, tables)[0]
    wide, _ = pa.rotary(k.float(), None, pos, rot)
    pa.kv_append_q8(wide, v.float().contiguous(), *want, clean, cl, st)
    lost = int(tables[0, 1])
    for a, b in zip(want, (*codes, *scales)):
        bits(a)[lost] = bits(b)[lost]
    got = pa.rotary_kv_append_q8(q, k, v, None, rot, *codes, *scales, bt, cl, st)
    with pytest.raises(pa.PagedAttnError) as e:
        pa.check_status()
    assert e.value.status == 5
    assert same_bits(got, pa.rotary(q, None, pos, rot)[0])
    for a, b in zip((*codes, *scales), want):
        assert same_bits(a, b)


def test_append_q8_starts_out_of_order(gpu):
    """A sequence that runs backwards is skipped and reported; one behind it
    that begins among an earlier one's units is still taken, as
    kv_append_q8 takes it."""
    rot, _ = rotary_of(pa, 64, gpu)
    lens = [80, 10, 40]
    starts = np.array([0, 80, 20, 60], dtype=np.int32)
    gen = np.random.default_rng(1)
    tables, nb = window_tables(lens, lens, 0, 0, gen)
    _, _, codes, scales = cache8(nb, 2, 64, 3, gpu)
    want = [t.clone() for t in (*codes, *scales)]
    q, k, v = projection(80, 4, 2, 64, "bf16", 3, gpu)
    pos = torch.from_numpy(gen.integers(0, 999, 80).astype(np.int32)).to(gpu)
    bt, cl, st = to_dev(gpu, tables, lens, starts)
    wide, _ = pa.rotary(k.float(), None, pos, rot)
    pa.kv_append_q8(wide, v.float().contiguous(), *want, bt, cl, st)
    with pytest.raises(pa.PagedAttnError):
        pa.check_status()
    got = pa.rotary_kv_append_q8(q, k, v, pos, rot, *codes, *scales, bt, cl, st)
    with pytest.raises(pa.PagedAttnError):
        pa.check_status()
    assert same_bits(got, pa.rotary(q, None, pos, rot)[0])
    for a, b in zip((*codes, *scales), want):
        assert same_bits(a, b)


def test_appends_on_two_streams_and_in_a_graph(gpu):
    rot, _ = rotary_of(pa, 128, gpu)
    qs, tables, nb, codes, scales = q8_case(gpu, 2, 128, 5)
    total = int(qs[-1])
    bt, cl, st = to_dev(gpu, tables, ALENS, qs)
    q, k, v = projection(total, 8, 2, 128, "f16", 3, gpu)
    pos = torch.from_numpy(places(ALENS, ANEW)).to(gpu)
    seq = np.repeat(np.arange(len(ALENS)), ANEW)
    slots = torch.from_numpy(tables[seq, places(ALENS, ANEW) // 16].astype(np.int64) * 16
                             + places(ALENS, ANEW) % 16).to(gpu)
    kc, vc = cache16(nb, 2, 128, "f16", 7, gpu)
    start = [t.clone() for t in (kc, vc, *codes, *scales)]
    q16 = pa.rotary_kv_append(q, k, v, pos, rot, kc, vc, slots)
    q8 = pa.rotary_kv_append_q8(q, k, v, None, rot, *codes, *scales, bt, cl, st)
    want = [t.clone() for t in (kc, vc, *codes, *scales)]
    a, b = torch.cuda.Stream(gpu), torch.cuda.Stream(gpu)

    def reset():
        for t, s in zip((kc, vc, *codes, *scales), start):
            bits(t).copy_(bits(s))

    def check(x, y):
        assert same_bits(x, q16) and same_bits(y, q8)
        for t, w in zip((kc, vc, *codes, *scales), want):
            assert same_bits(t, w)

    reset()
    main = torch.cuda.current_stream(gpu)
    a.wait_stream(main)
    b.wait_stream(main)
    x = pa.rotary_kv_append(q, k, v, pos, rot, kc, vc, slots, stream=a)
    y = pa.rotary_kv_append_q8(q, k, v, None, rot, *codes, *scales, bt, cl, st, stream=b)
    main.wait_stream(a)
    main.wait_stream(b)
    check(x, y)
    graph = torch.cuda.CUDAGraph()
    x, y = torch.empty_like(q16), torch.empty_like(q8)
    with torch.cuda.graph(graph):
        pa.rotary_kv_append(q, k, v, pos, rot, kc, vc, slots, q_out=x)
        pa.rotary_kv_append_q8(q, k, v, None, rot, *codes, *scales, bt, cl, st, q_out=y)
    for _ in range(2):
        reset()
        graph.replay()
        check(x, y)
    pa.check_status()


def test_many_tokens(gpu):
    """A chunk of thousands of tokens over ragged sequences, both caches."""
    rot, _ = rotary_of(pa, 128, gpu, base=500000.0)
    gen = np.random.default_rng(2)
    lens = gen.integers(1, 3000, 23)
    new = np.minimum(gen.integers(1, 900, 23), lens)
    qs, tables, nb, codes, scales = q8_case(gpu, 8, 128, 3, lens, new)
    total = int(qs[-1])
    where = places(lens, new)
    pos = torch.from_numpy(where).to(gpu)
    bt, cl, st = to_dev(gpu, tables, lens, qs)
    q, k, v = projection(total, 32, 8, 128, "bf16", 3, gpu)
    qo, ko = pa.rotary(q, k, pos, rot)
    wide, _ = pa.rotary(k.float(), None, pos, rot)
    want = [t.clone() for t in (*codes, *scales)]
    pa.kv_append_q8(wide, v.float().contiguous(), *want, bt, cl, st)
    assert same_bits(pa.rotary_kv_append_q8(q, k, v, None, rot, *codes, *scales, bt, cl, st), qo)
    for t, w in zip((*codes, *scales), want):
        assert same_bits(t, w)
    kc, vc = cache16(nb, 8, 128, "bf16", 7, gpu)
    kw, vw = kc.clone(), vc.clone()
    seq = np.repeat(np.arange(len(lens)), new)
    slots = torch.from_numpy(tables[seq, where // 16].astype(np.int64) * 16 + where % 16).to(gpu)
    pa.kv_append(ko, v.contiguous(), kw, vw, slots)
    assert same_bits(pa.rotary_kv_append(q, k, v, pos, rot, kc, vc, slots), qo)
    assert same_bits(kc, kw) and same_bits(vc, vw)
    pa.check_status()
