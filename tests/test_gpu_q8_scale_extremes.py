"""8-bit decode with value scales at the ends of their range, very uneven
within a sequence and from one sequence to the next: each output is held to a
bound made from its own sequence's and head's weights and scales, so that an
output of zeros, or one whose small blocks are lost, fails.

The bound, for one (sequence, head), with p_t the softmax's weights, s_t the
scale of t's block and c_t its codes, out = sum p_t s_t c_t:
  - the output's rounding, half a step (f16 below its normal range: 2^-25);
  - scores: 132 half steps of 32 bits relative to ``size``, twice in exp, and 2
    more steps of exp itself; sums of a score with a scale's exponent (up to
    2^7, so half a step is 2^-18), three of them, in a power of two: 2^-16
    relative;
  - p_t s_t rounded to f16: half a step, or where the product is subnormal
    2^-25 of the f16 number 1, which is at most 2^-7 of max_t p_t s_t: per
    token 2^-32 max p s |c_t|, |c_t| <= 448;
  - fp32 sums of n terms, numerator and denominator, half a step each, as much
    again for rescaling and merging.
"""

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from oracle import cache_q8 as oq
from oracle import windowed as ow
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.gpu_helpers import TORCH_DTYPES, to_f32_numpy
from tests.test_gpu_q8 import Mirror
from tests.test_gpu_window import to_dev
from tests.window_helpers import HALF_STEP, window_tables

pytestmark = pytest.mark.gpu


def reference(q, codes, scales, tables, lens, window, sinks, scale, out_type):
    """(out, limit), both [B, Hq, d] in 64 bits."""
    values = [oq.decode(c) for c in codes]
    hkv = codes[0].shape[1]
    u = HALF_STEP["f32"]
    out, limit = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(len(lens)):
        tokens = ow.visible_tokens(int(lens[b]) - 1, window, sinks)
        n = len(tokens)
        for g in range(hkv):
            k = ow.gather_tokens(values[0], tables[b], tokens, g, scales[0])
            c = ow.gather_tokens(values[1], tables[b], tokens, g)
            s = np.array([float(scales[1][tables[b][t // 16], g]) for t in tokens])
            for h in range(g * (q.shape[1] // hkv), (g + 1) * (q.shape[1] // hkv)):
                x = scale * (k @ q[b, h].astype(np.float64))
                p = np.exp(x - x.max())
                p /= p.sum()
                size = abs(scale) * float((np.abs(k) @ np.abs(q[b, h])).max())
                out[b, h] = (p * s) @ c
                spread = (p * s) @ np.abs(c)
                rel = 2 * 132 * u * size + 8 * u + 2.0 ** -16 + 4 * n * u + HALF_STEP["f16"]
                limit[b, h] = (HALF_STEP[out_type] * np.abs(out[b, h]) + rel * spread) * (1 + 2.0 ** -7) \
                    + n * 2.0 ** -32 * (p * s).max() * 448 + (2.0 ** -25 if out_type == "f16" else 0)
    return out, limit


RANGES = [
    [(-100, -97), (117, 120), (0, 1), (-60, -57)],            # a range of its own per sequence
    [(-100, 110), (-100, -60), (60, 110), (-3, 4)],           # and very uneven ones
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 20)])
@pytest.mark.parametrize("ranges", RANGES, ids=["apart", "mixed"])
def test_decode_is_right_at_every_scale(gpu, dtype, head_dim, window, sinks, ranges):
    lens = [300, 47, 600, 16]
    gen = np.random.default_rng(37 + head_dim)
    tables, nb = window_tables(lens, lens, 0, 0, gen)
    m = Mirror(nb, 2, head_dim, 41, gpu)
    if dtype == "f16":                       # within what an f16 output holds: 448 * 2^6 at most
        ranges = [(max(-20, min(a, 4)), max(-19, min(b, 6))) for a, b in ranges]
    m.scales[0][:] = np.exp2(gen.integers(-12, -6, m.scales[0].shape))
    for b, (low, high) in enumerate(ranges):
        held = tables[b][: (lens[b] + 15) // 16]
        m.scales[1][held] = np.exp2(gen.integers(low, high, (len(held), 2)))
    for i in range(2):
        m.dscales[i].copy_(torch.from_numpy(m.scales[i]))
    q = wl.normal((4, 8, head_dim), TORCH_DTYPES[dtype], 43, gpu)
    bt, cl = to_dev(gpu, tables, lens)
    out = pa.paged_attention_decode_q8(q, *m.dcodes, *m.dscales, bt, cl, window, sinks, head_dim ** -0.5)
    pa.check_status()
    want, limit = reference(to_f32_numpy(q), m.codes, m.scales, tables, lens, window, sinks,
                            head_dim ** -0.5, dtype)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    over = np.abs(got - want) - limit
    assert (over <= 0).all(), f"{int((over > 0).sum())} outside, worst {np.max(np.abs(got - want) / limit):.2f} of the bound"
    # the bound itself tells right from wrong: for most outputs of every
    # sequence it is far under the value
    for b in range(4):
        assert np.mean(limit[b] < 0.1 * np.abs(want[b])) > 0.8



@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("exponent", [-100, 117])
def test_sums_and_scales_together(gpu, head_dim, exponent):
    """The softmax's sum and the value scales lie at opposite ends of 32 bits'
    range, or at the same one; the outputs are ordinary numbers of the scales'
    size.  700 sequences of 3200 tokens that share their blocks: most (sequence,
    head) runs are one warp's, whose references stay at the first block's score,
    7.9 bits (under 8) below all others.

    Every query is (1, 0, ..), the first block's keys are 0 and all others 16 * 2^-4
    in column 0, so the scores are 0 and ``scale``.  The bound: the output's half
    step; weights rounded to f16, half a step; 3200 / 16 terms and 64 more of merges
    in 32 bits, twice; 2^-16 for exponents of 2^7; scores of 8 off by 2^-20."""
    hkv, hq, n, batch = 8, 16, 3200, 700
    nb = n // 16
    gen = np.random.default_rng(3)
    scale = float(np.float32(7.9 / np.log2(np.e)))
    k = np.zeros((nb, hkv, 16, head_dim))
    k[1:, :, :, 0] = 16
    v = 1 + gen.integers(0, 8, k.shape) / 8.0
    codes = [torch.from_numpy(oq.encode(x)).to(gpu).view(torch.float8_e4m3fn) for x in (k, v)]
    scales = [torch.full((nb, hkv), s, device=gpu) for s in (2.0 ** -4, 2.0 ** exponent)]
    tables = np.tile(np.arange(nb, dtype=np.int32), (batch, 1))
    q = torch.zeros((batch, hq, head_dim), dtype=torch.bfloat16, device=gpu)
    q[..., 0] = 1
    bt, cl = to_dev(gpu, tables, [n] * batch)
    out = pa.paged_attention_decode_q8(q, *codes, *scales, bt, cl, 0, 0, scale)
    pa.check_status()
    w = np.where(np.arange(nb) == 0, 2.0 ** -7.9, 1.0)[:, None, None, None]
    want = ((w * v).sum((0, 2)) / (16 * w.sum()) * 2.0 ** exponent).repeat(2, axis=0)       # [hq, d]
    rel = HALF_STEP["bf16"] + HALF_STEP["f16"] + 2 * (n / 16 + 64) * HALF_STEP["f32"] + 2.0 ** -16 + 2.0 ** -20
    err = np.abs(out.double().cpu().numpy() / want - 1)
    assert err.max() <= rel * (1 + 2.0 ** -7), f"worst {err.max():.2e} of the value, allowed {rel:.2e}"
