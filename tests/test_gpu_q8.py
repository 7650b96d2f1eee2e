"""The 8-bit cache on the GPU: quantising append and reading back are exact
against the oracle, decode is within the roundings' bound, and a prompt and
decode steps run through all of them together."""

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from oracle import cache_q8 as oq
from oracle import windowed as ow
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.gpu_helpers import TORCH_DTYPES, to_f32_numpy
from tests.test_gpu_window import to_dev
from tests.window_helpers import assert_within, bound, cache8, window_tables

pytestmark = pytest.mark.gpu


def codes_of(t):
    return t.view(torch.uint8).cpu().numpy()


class Mirror:
    """A device cache and the oracle's copy of it."""

    def __init__(self, nb, hkv, d, seed, dev, spread=3):
        self.codes, self.scales, self.dcodes, self.dscales = cache8(nb, hkv, d, seed, dev, spread)

    def append(self, k, v, tables, lens, qs, dev):
        bt, cl, st = to_dev(dev, tables, lens, qs)
        pa.kv_append_q8(k, v, *self.dcodes, *self.dscales, bt, cl, st)
        oq.kv_append_q8(to_f32_numpy(k), to_f32_numpy(v), *self.codes, *self.scales, tables, lens, qs)

    def check(self):
        for i in range(2):
            np.testing.assert_array_equal(self.dscales[i].cpu().numpy(), self.scales[i])
            got, want = codes_of(self.dcodes[i]), self.codes[i]
            nan = (got & 0x7F) == 0x7F
            np.testing.assert_array_equal(nan, (want & 0x7F) == 0x7F)
            np.testing.assert_array_equal(got[~nan], want[~nan])


ALENS = [1, 16, 17, 40, 64, 100, 33, 5, 200, 18]
ANEW = [1, 16, 3, 24, 0, 100, 1, 5, 77, 1]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("hkv", [1, 5, 8])
def test_append_is_exact(gpu, dtype, head_dim, hkv):
    """Codes, scales and every byte that must stay, over chunks that begin and
    end anywhere in a block, growing scales among them."""
    gen = np.random.default_rng(hkv + head_dim)
    qs = np.concatenate([[0], np.cumsum(ANEW)])
    tables, nb = window_tables(ALENS, ALENS, 0, 0, gen)
    m = Mirror(nb, hkv, head_dim, 7, gpu)
    g = torch.Generator(device=gpu).manual_seed(5)
    for step in range(3):
        k, v = (torch.randn((int(qs[-1]), hkv, head_dim), generator=g, device=gpu)
                * torch.exp(2 * torch.randn((int(qs[-1]), hkv, 1), generator=g, device=gpu))
                for _ in range(2))
        m.append(k.to(TORCH_DTYPES[dtype]), v.to(TORCH_DTYPES[dtype]), tables, ALENS, qs, gpu)
        m.check()
    pa.check_status()


def test_append_special_values(gpu):
    """Zeros, subnormals, the type's largest, infinities and NaN; scales at
    both ends of their range."""
    rows = torch.zeros((12, 1, 64), device=gpu)
    rows[1] = 1e-38
    rows[2] = 3e38
    rows[3, 0, :3] = torch.tensor([float("inf"), -float("inf"), float("nan")])
    rows[4] = float("nan")
    rows[5] = float("inf")
    rows[6, 0, 0], rows[6, 0, 1] = 448.0, -448.1
    rows[7] = -0.0
    rows[8] = torch.linspace(-500, 500, 64)
    rows[9] = 2.0 ** -100
    rows[10] = 1.75
    rows[11] = 1.7500001
    for dtype in ("f32", "bf16"):
        k = rows.to(TORCH_DTYPES[dtype])
        tables = np.arange(12, dtype=np.int32)[:, None]
        m = Mirror(13, 1, 64, 3, gpu)
        m.append(k, -k, tables, [1] * 12, list(range(13)), gpu)       # a block each, fresh
        m.check()
        m.append(k.flip(0), k, tables, [2] * 12, list(range(13)), gpu)  # held token, new scale
        m.check()
        m.append(k, k, np.array([[12]], dtype=np.int32), [12], [0, 12], gpu)   # all in one block
        m.check()
    pa.check_status()


def test_append_token_by_token(gpu):
    """A hundred decode steps of a ragged batch, the scales growing as they
    go: bit for bit the oracle's at every step."""
    gen = np.random.default_rng(17)
    lens = np.array([1, 15, 16, 17, 40])
    tables, nb = window_tables(lens + 100, lens + 100, 0, 0, gen)
    m = Mirror(nb, 2, 128, 11, gpu)
    g = torch.Generator(device=gpu).manual_seed(3)
    for step in range(100):
        size = torch.exp(1.5 * torch.randn((5, 2, 1), generator=g, device=gpu))
        k, v = ((torch.randn((5, 2, 128), generator=g, device=gpu) * size).bfloat16() for _ in range(2))
        m.append(k, v, tables, lens + step, list(range(6)), gpu)
        if step % 9 == 0 or step > 95:
            m.check()
    pa.check_status()


def test_append_many_sequences(gpu):
    """More sequences than a thread block has threads, most of them idle or
    with a token or two."""
    gen = np.random.default_rng(21)
    new = np.minimum(gen.integers(0, 4, 700), 2)
    new[[3, 400, 699]] = [40, 17, 100]
    lens = new + gen.integers(0, 40, 700)
    tables, nb = window_tables(lens, lens, 0, 0, gen)
    qs = np.concatenate([[0], np.cumsum(new)])
    m = Mirror(nb, 2, 64, 15, gpu)
    k, v = (wl.normal((int(qs[-1]), 2, 64), torch.bfloat16, 17 + i, gpu) * 3 for i in range(2))
    m.append(k, v, tables, lens, qs, gpu)
    m.check()
    pa.check_status()


def test_append_bad_input(gpu):
    """Bad lengths, rows and table entries skip what they concern, set the
    status and change nothing else."""
    gen = np.random.default_rng(19)
    tables, nb = window_tables([20, 20, 20], [20] * 3, 0, 0, gen)
    k = wl.normal((9, 2, 64), torch.float16, 5, gpu)
    good = Mirror(nb, 2, 64, 13, gpu)
    good.append(k, k, tables, [20, 20, 20], [0, 3, 6, 9], gpu)
    good.check()
    for lens, qs, tab in (([2, 20, 20], [0, 3, 6, 9], None), ([40, 20, 20], [0, 3, 6, 9], None),
                          ([20, 20, 20], [0, 3, 6, 10], None), ([20, 20, 20], [-1, 3, 6, 9], None),
                          ([20, 20, 20], [0, 6, 3, 9], None), ([20, 20, 20], [0, 3, 6, 9], -1),
                          ([20, 20, 20], [0, 3, 6, 9], nb)):
        m = Mirror(nb, 2, 64, 13, gpu)
        t = tables.copy()
        if tab is not None:
            t[0, 1] = tab
        bt, cl, st = to_dev(gpu, t, lens, qs)
        pa.kv_append_q8(k, k, *m.dcodes, *m.dscales, bt, cl, st)
        with pytest.raises(pa.PagedAttnError) as e:
            pa.check_status()
        assert e.value.status == 5
        # the sequences that are in order, each by itself (a bad entry's block
        # is the only one its sequence's three tokens touch)
        for b in range(3):
            q0, q1, n = qs[b], qs[b + 1], lens[b]
            if 0 <= q0 <= q1 <= 9 and q1 - q0 <= n <= t.shape[1] * 16 and 0 <= t[b, 1] < nb:
                rows = to_f32_numpy(k)[q0:q1]
                oq.kv_append_q8(rows, rows, *m.codes, *m.scales, t[b:b + 1], [n], [0, q1 - q0])
        m.check()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hkv,head_dim", [(1, 64), (3, 128), (8, 128), (32, 64)])
def test_dequantize_is_exact(gpu, dtype, hkv, head_dim):
    m = Mirror(9, hkv, head_dim, 23, gpu, spread=4)
    pairs = np.array([[3, 0], [8, 5], [0, 2], [3, 4]], dtype=np.int64)
    out = [torch.full((6, hkv, 16, head_dim), 9.0, dtype=TORCH_DTYPES[dtype], device=gpu) for _ in range(2)]
    pa.block_dequantize(*m.dcodes, *m.dscales, torch.from_numpy(pairs).to(gpu), *out)
    pa.check_status()
    for i in range(2):
        want = np.full((6, hkv, 16, head_dim), 9.0)
        oq.block_dequantize(m.codes[i], m.scales[i], pairs, want)
        want = torch.from_numpy(want).to(TORCH_DTYPES[dtype])
        assert torch.equal(out[i].cpu(), want)
    bad = torch.tensor([[9, 0], [0, 6], [-1, 1], [1, 1]], device=gpu)
    pa.block_dequantize(*m.dcodes, *m.dscales, bad, *out)
    with pytest.raises(pa.PagedAttnError) as e:
        pa.check_status()
    assert e.value.status == 5
    want = oq.decode(m.codes[0][1]) * m.scales[0][1].astype(np.float64)[:, None, None]
    assert torch.equal(out[0][1].cpu(), torch.from_numpy(want).to(TORCH_DTYPES[dtype]))
    assert torch.equal(out[0][0].cpu(), torch.from_numpy(
        oq.decode(m.codes[0][3]) * m.scales[0][3].astype(np.float64)[:, None, None]).to(TORCH_DTYPES[dtype]))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_dequantize_into_unaligned_sectors(gpu, dtype):
    """Outputs that begin 16 bytes past a 32-byte boundary."""
    m = Mirror(4, 2, 64, 25, gpu)
    t = TORCH_DTYPES[dtype]
    skip = 16 // t.itemsize
    n = 3 * 2 * 16 * 64
    out = [torch.zeros(n + 2 * skip, dtype=t, device=gpu)[skip:skip + n].view(3, 2, 16, 64) for _ in range(2)]
    assert out[0].data_ptr() % 32 == 16
    pairs = torch.tensor([[2, 0], [0, 1], [3, 2]], device=gpu)
    pa.block_dequantize(*m.dcodes, *m.dscales, pairs, *out)
    pa.check_status()
    for i in range(2):
        want = torch.stack([m.dcodes[i].float()[j] * m.dscales[i][j][:, None, None] for j in (2, 0, 3)])
        assert torch.equal(out[i], want.to(t))


# -------------------------------------------------------------------- decode
def check_decode(out, q, m, tables, lens, window, sinks, dtype, rows=None, scale=None):
    d = q.shape[2]
    values = [oq.decode(c) for c in m.codes]
    ref, spread, size = ow.decode(to_f32_numpy(q), *values, tables, lens, window, sinks,
                                  d ** -0.5 if scale is None else scale, *m.scales, rows=rows)
    tokens = min(int(max(lens)), window + sinks) if window else int(max(lens))
    # the weights are rounded no more coarsely than to f16; the queries not at all
    assert_within(out, ref, bound(ref, spread, size, tokens, dtype, "f16",
                                  448.0 * float(m.scales[1].max())))


LENS = [0, 1, 15, 16, 17, 33, 100, 257, 530, 1999]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("heads", [(8, 8), (32, 8), (10, 2), (16, 2)], ids=["g1", "g4", "g5", "g8"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 4), (129, 40)])
def test_decode_matches_oracle(gpu, dtype, head_dim, heads, window, sinks):
    hq, hkv = heads
    gen = np.random.default_rng(hq + window)
    tables, nb = window_tables(LENS, [1] * len(LENS), window, sinks, gen)
    m = Mirror(nb, hkv, head_dim, 29 + hq, gpu)
    q = wl.normal((len(LENS), hq, head_dim), TORCH_DTYPES[dtype], 31 + window, gpu)
    bt, cl = to_dev(gpu, tables, LENS)
    out = pa.paged_attention_decode_q8(q, *m.dcodes, *m.dscales, bt, cl, window, sinks, head_dim ** -0.5)
    pa.check_status()
    check_decode(out, q, m, tables, LENS, window, sinks, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("low,high", [(-100, -90), (-20, 0), (-60, -8), (-7, 110)])
def test_decode_uneven_scales(gpu, dtype, low, high):
    """Scales of very different size from block to block: the values' scales
    as they come, the keys' small enough that the scores stay ordinary."""
    gen = np.random.default_rng(37)
    lens = [300, 47, 16]
    tables, nb = window_tables(lens, lens, 0, 0, gen)
    m = Mirror(nb, 2, 128, 41, gpu)
    if dtype == "f16":
        high = min(high, 4)
        low = min(low, high - 8)
    m.scales[0][:] = np.exp2(gen.integers(-12, -6, m.scales[0].shape))
    m.scales[1][:] = np.exp2(gen.integers(low, high, m.scales[1].shape))
    for i in range(2):
        m.dscales[i].copy_(torch.from_numpy(m.scales[i]))
    q = wl.normal((3, 8, 128), TORCH_DTYPES[dtype], 43, gpu)
    bt, cl = to_dev(gpu, tables, lens)
    out = pa.paged_attention_decode_q8(q, *m.dcodes, *m.dscales, bt, cl, 0, 0, 128 ** -0.5)
    pa.check_status()
    check_decode(out, q, m, tables, lens, 0, 0, dtype)


@pytest.mark.parametrize("size", [1e-30, 1e-6, 3e4, 1e20])
def test_decode_queries_of_any_size(gpu, size):
    """bf16 queries far outside f16's range, with a softmax scale to match."""
    gen = np.random.default_rng(47)
    tables, nb = window_tables([200, 31], [1, 1], 0, 0, gen)
    m = Mirror(nb, 2, 64, 53, gpu)
    q = (wl.normal((2, 8, 64), torch.float32, 59, gpu) * size).bfloat16()
    q[1, 3] = 0
    bt, cl = to_dev(gpu, tables, [200, 31])
    scale = 0.125 / size
    out = pa.paged_attention_decode_q8(q, *m.dcodes, *m.dscales, bt, cl, 0, 0, scale)
    pa.check_status()
    check_decode(out, q, m, tables, [200, 31], 0, 0, "bf16", scale=float(np.float32(scale)))


@pytest.mark.parametrize("window,sinks", [(0, 0), (37, 5)])
def test_decode_masked_slots_may_hold_anything(gpu, window, sinks):
    lens = np.array([200, 41, 64, 90, 1])
    gen = np.random.default_rng(61)
    tables, nb = window_tables(lens, lens, 0, 0, gen)
    m = Mirror(nb + 2, 2, 128, 67, gpu)
    q = wl.normal((5, 8, 128), torch.bfloat16, 71, gpu)
    bt, cl = to_dev(gpu, tables, lens)
    clean = pa.paged_attention_decode_q8(q, *m.dcodes, *m.dscales, bt, cl, window, sinks, 0.09)
    keep = torch.zeros((nb + 2, 16), dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in ow.visible_tokens(int(n) - 1, window, sinks):
            keep[int(tables[b, t // 16]), t % 16] = True
    hide = ~keep.to(gpu)[:, None, :, None].expand_as(m.dcodes[0])
    for bad in (0x7F, 0xFF, 0x7E, 0xFE):
        dirty = [c.view(torch.uint8).masked_fill(hide, bad).view(torch.float8_e4m3fn) for c in m.dcodes]
        unseen = ~keep.any(1).to(gpu)
        scales = [s.masked_fill(unseen[:, None], float("nan")) for s in m.dscales]
        out = pa.paged_attention_decode_q8(q, *dirty, *scales, bt, cl, window, sinks, 0.09)
        assert torch.equal(out, clean)
    pa.check_status()


def test_decode_many_and_long(gpu):
    gen = np.random.default_rng(73)
    lens = np.concatenate([gen.integers(0, 60, 500), [20000, 12345], gen.integers(0, 60, 200)])
    tables, nb = window_tables(lens, [1] * len(lens), 0, 0, gen)
    m = Mirror(nb, 4, 128, 79, gpu)
    q = wl.normal((len(lens), 8, 128), torch.bfloat16, 83, gpu)
    bt, cl = to_dev(gpu, tables, lens)
    out = pa.paged_attention_decode_q8(q, *m.dcodes, *m.dscales, bt, cl, 0, 0, 128 ** -0.5)
    again = pa.paged_attention_decode_q8(q, *m.dcodes, *m.dscales, bt, cl, 0, 0, 128 ** -0.5)
    pa.check_status()
    assert torch.equal(out, again)
    check_decode(out, q, m, tables, lens, 0, 0, "bf16", rows={0, 250, 499, 500, 501, 502, 701})


@pytest.mark.parametrize("head_dim", [64, 128])
def test_decode_one_sequence_over_every_sm(gpu, head_dim):
    gen = np.random.default_rng(75)
    tables, nb = window_tables([70001], [1], 0, 0, gen)
    m = Mirror(nb, 1, head_dim, 77, gpu)
    q = wl.normal((1, 8, head_dim), torch.bfloat16, 85, gpu)
    bt, cl = to_dev(gpu, tables, [70001])
    out = pa.paged_attention_decode_q8(q, *m.dcodes, *m.dscales, bt, cl, 0, 0, head_dim ** -0.5)
    pa.check_status()
    check_decode(out, q, m, tables, [70001], 0, 0, "bf16")


@pytest.mark.parametrize("hkv,head_dim", [(2, 64), (4, 128)])
def test_forked_sequences_copy_on_write(gpu, hkv, head_dim):
    """A fork of a sequence in an 8-bit cache: the shared last block is copied
    (block_copy over the codes viewed as 16-bit elements, the scales by
    index), then both branches append and decode."""
    hq = 2 * hkv
    m = Mirror(12, hkv, head_dim, 121, gpu)
    tables = np.array([[3, 7, 1], [3, 7, 5]], dtype=np.int32)
    prompt = wl.normal((40, hkv, head_dim), torch.bfloat16, 123, gpu)
    m.append(prompt, prompt, tables[:1], [40], [0, 40], gpu)
    as16 = [c.view(torch.uint8).view(12, -1).view(torch.float16).view(12, -1, 16, 64) for c in m.dcodes]
    pa.block_copy(as16[:1], as16[1:], torch.tensor([[1, 5]], device=gpu))
    for i in range(2):
        m.dscales[i][5] = m.dscales[i][1]
        m.codes[i][5], m.scales[i][5] = m.codes[i][1], m.scales[i][1]
    m.check()
    for step in range(4):
        lens = np.array([41 + step, 41 + step])
        k, v = (wl.normal((2, hkv, head_dim), torch.bfloat16, 125 + 2 * step + i, gpu) * 2.0 ** step
                for i in range(2))
        m.append(k, v, tables, lens, [0, 1, 2], gpu)
        m.check()
        q = wl.normal((2, hq, head_dim), torch.bfloat16, 141 + step, gpu)
        bt, cl = to_dev(gpu, tables, lens)
        out = pa.paged_attention_decode_q8(q, *m.dcodes, *m.dscales, bt, cl, 0, 0, 0.1)
        pa.check_status()
        check_decode(out, q, m, tables, lens, 0, 0, "bf16", scale=0.1)


def test_decode_scale_of_zero(gpu):
    """A block whose scale is zero holds zeros: it keeps its share of the
    softmax (its scores are 0) and adds nothing."""
    gen = np.random.default_rng(143)
    tables, nb = window_tables([60, 20], [1, 1], 0, 0, gen)
    m = Mirror(nb, 2, 128, 145, gpu)
    for i in range(2):
        m.scales[i][tables[0, 1]] = 0
        m.scales[i][tables[1, :2]] = 0
        m.dscales[i].copy_(torch.from_numpy(m.scales[i]))
    q = wl.normal((2, 8, 128), torch.bfloat16, 147, gpu)
    bt, cl = to_dev(gpu, tables, [60, 20])
    out = pa.paged_attention_decode_q8(q, *m.dcodes, *m.dscales, bt, cl, 0, 0, 128 ** -0.5)
    pa.check_status()
    check_decode(out, q, m, tables, [60, 20], 0, 0, "bf16")
    assert (out[1] == 0).all()


def test_q8_cache_past_32_bit_offsets(gpu):
    nb = (1 << 32) // (8 * 16 * 128) + 64
    m = Mirror(40, 8, 128, 89, gpu)
    big = [torch.zeros((nb, 8, 16, 128), dtype=torch.uint8, device=gpu).view(torch.float8_e4m3fn)
           for _ in range(2)]
    scales = [torch.ones((nb, 8), device=gpu) for _ in range(2)]
    for i in range(2):
        big[i].view(torch.uint8)[-40:] = m.dcodes[i].view(torch.uint8)
        scales[i][-40:] = m.dscales[i]
    tables = (nb - 1 - np.arange(40)[None]).astype(np.int32)
    bt, cl, st = to_dev(gpu, tables, [635], [0, 30])
    low = bt - (nb - 40)
    k = wl.normal((30, 8, 128), torch.bfloat16, 97, gpu)
    pa.kv_append_q8(k, k, *big, *scales, bt, cl, st)
    pa.kv_append_q8(k, k, *m.dcodes, *m.dscales, low, cl, st)
    q = wl.normal((1, 32, 128), torch.bfloat16, 101, gpu)
    a = pa.paged_attention_decode_q8(q, *big, *scales, bt, cl, 0, 0, 0.1)
    b = pa.paged_attention_decode_q8(q, *m.dcodes, *m.dscales, low, cl, 0, 0, 0.1)
    out = [torch.empty((1, 8, 16, 128), device=gpu) for _ in range(2)]
    pa.block_dequantize(*big, *scales, torch.tensor([[nb - 1, 0]], device=gpu), *out)
    pa.check_status()
    assert torch.equal(a, b)
    assert torch.equal(out[0][0], m.dcodes[0][39].float() * m.dscales[0][39][:, None, None])


def test_shared_plan_and_captured_step(gpu):
    """A decode step as a serving loop runs it, captured: append, then one plan
    for several layers' 8-bit decodes, replayed as the sequences grow."""
    hq, hkv, d, window, sinks, layers = 32, 8, 128, 64, 4, 3
    gen = np.random.default_rng(103)
    lens = np.array([90, 16, 31, 200])
    tables, nb = window_tables(lens + 20, lens + 20, 0, 0, gen)
    mirrors = [Mirror(nb, hkv, d, 107 + i, gpu) for i in range(layers)]
    bt, cl, st = to_dev(gpu, tables, lens, range(5))
    k, v = (torch.zeros((4, hkv, d), dtype=torch.bfloat16, device=gpu) for _ in range(2))
    q = torch.zeros((4, hq, d), dtype=torch.bfloat16, device=gpu)
    outs = [torch.zeros_like(q) for _ in range(layers)]
    mb = tables.shape[1]
    ws = pa.alloc_window_workspace(4, hq, hkv, d, mb, gpu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.paged_attention_decode_window_plan(cl, window, sinks, hq, hkv, d, mb, ws)
        for m, out in zip(mirrors, outs):
            pa.kv_append_q8(k, v, *m.dcodes, *m.dscales, bt, cl, st)
            pa.paged_attention_decode_q8_run(q, *m.dcodes, *m.dscales, bt, cl, window, sinks,
                                             d ** -0.5, ws, out=out)
    for step in range(1, 20):
        lens = lens + 1
        cl += 1
        for i, t in enumerate((k, v, q)):
            t.copy_(wl.normal(t.shape, t.dtype, 1000 * step + i, gpu))
        graph.replay()
        torch.cuda.synchronize()
        for m, out in zip(mirrors, outs):
            oq.kv_append_q8(to_f32_numpy(k), to_f32_numpy(v), *m.codes, *m.scales, tables, lens, range(5))
            if step % 6 == 1:
                m.check()
                check_decode(out, q, m, tables, lens, window, sinks, "bf16")
    pa.check_status()


@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 4)])
def test_prompts_then_decode(gpu, window, sinks):
    """Chunked prompts and decode steps over an 8-bit cache, with blocks behind
    the window freed and used again: append, read the visible blocks back,
    prefill over them, then append and decode."""
    hq, hkv, d, dtype = 8, 2, 128, torch.bfloat16
    lens = np.zeros(3, dtype=np.int64)
    chunks = [np.array(c) for c in ([50, 16, 1], [30, 100, 0], [0, 33, 90], [1, 1, 1], [1, 1, 1])]
    total = sum(chunks)
    width = int((total.max() + 15) // 16)
    nb = 40
    free = list(np.random.default_rng(109).permutation(nb))
    tables = np.full((3, width), -1, dtype=np.int32)
    m = Mirror(nb, hkv, d, 113, gpu)
    for step, new in enumerate(chunks):
        lens = lens + new
        for b in range(3):
            for blk in range(width):
                seen = blk * 16 < lens[b]
                if window and blk * 16 >= sinks:
                    seen &= (blk + 1) * 16 > lens[b] - new[b] - window + 1
                if seen and tables[b, blk] < 0:
                    tables[b, blk] = free.pop()
                elif not seen and tables[b, blk] >= 0:
                    free.insert(0, tables[b, blk])
                    tables[b, blk] = -1
        qs = np.concatenate([[0], np.cumsum(new)])
        k, v = (wl.normal((int(qs[-1]), hkv, d), dtype, 127 + 10 * step + i, gpu) for i in range(2))
        q = wl.normal((int(qs[-1]), hq, d), dtype, 131 + step, gpu)
        m.append(k, v, tables, lens, qs, gpu)
        m.check()
        bt, cl, st = to_dev(gpu, tables, lens, qs)
        values = [oq.decode(c) for c in m.codes]
        ref, spread, size = ow.prefill(to_f32_numpy(q), *values, tables, lens, qs, window, sinks,
                                       d ** -0.5, *m.scales)
        if new.max() > 1:
            held = tables[tables >= 0].astype(np.int64)
            pairs = torch.from_numpy(np.stack([held, np.arange(len(held))], 1)).to(gpu)
            staged = np.where(tables >= 0, 0, -1)
            staged[tables >= 0] = np.arange(len(held))
            k16, v16 = (torch.empty((len(held), hkv, 16, d), dtype=dtype, device=gpu) for _ in range(2))
            pa.block_dequantize(*m.dcodes, *m.dscales, pairs, k16, v16)
            out = pa.paged_attention_prefill_window(q, k16, v16, to_dev(gpu, staged)[0], cl, st,
                                                    window, sinks, d ** -0.5)
        else:
            out = pa.paged_attention_decode_q8(q, *m.dcodes, *m.dscales, bt, cl, window, sinks, d ** -0.5)
        pa.check_status()
        assert_within(out, ref, bound(ref, spread, size, int(lens.max()), "bf16", "bf16"))
