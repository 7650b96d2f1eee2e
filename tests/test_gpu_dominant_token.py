"""A first token that takes most of the softmax, with many others sharing the
rest: the small weights must keep their share when they are rounded to 16 bits
for the product with V.

Every query is (1, 0, ..), every key but the first is zero and the first is
(16, 0, ..), so that all other weights are 2^-bits of the first one's, bits =
scale * 16 * log2 e; the first value row is zero, so the output is the small
weights' part alone and any loss of theirs is seen whole.  (Keys, queries and
scores are exact in every type; log2 e in 32 bits moves a score by less than
2^-18, its weight by less than 2^-18 of itself.)

The bound.  A weight w = 2^-bits of the largest is stored as w * 2^L rounded
to f16, L the factor the kernels lift weights by: half a step of f16 is
2^-11 relative, or 2^-25 absolute where w * 2^L is subnormal.  The reference
may be the largest score itself, so nothing is gained from it, and L >= 7.
Relative to the output (its terms are all positive): 2^-11 + 2^-25-L+bits.
fp32 sums: a run of n tokens is added up 16 at a time, n / 16 terms per warp
at most, each a half step: 2 (n / 16 + 64) 2^-24 for numerator and
denominator, 64 of merges and the rest.  2^-17 for the scores.  The output's
own rounding: half a step, and 2^-25 absolute below f16's normal range.
"""

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from oracle import cache_q8 as oq
from tests.gpu_helpers import TORCH_DTYPES
from tests.test_gpu_window import to_dev
from tests.window_helpers import HALF_STEP

pytestmark = pytest.mark.gpu

LIFT = 7
BITS = [14.5, 20.4, 23.46, 25.5, 27.3]


def scale_for(bits):
    return float(np.float32(bits / (16 * np.log2(np.e))))


def cache(nb, hkv, d, seed):
    """Keys and values [nb, hkv, 16, d] in 64 bits; block 0 begins with the
    dominant token.  Values are e4m3's own, between 1 and 1.875."""
    gen = np.random.default_rng(seed)
    k = np.zeros((nb, hkv, 16, d))
    k[0, :, 0, 0] = 16.0
    v = 1 + gen.integers(0, 8, k.shape) / 8.0
    v[0, :, 0] = 0
    return k, v


def expected(v, tables, seen, bits):
    """out [B, hkv, d]: the values of the tokens seen (a list per sequence;
    token 0 first), weighted."""
    out = []
    w = 2.0 ** -bits
    for b, tokens in enumerate(seen):
        rows = v[tables[b][tokens // 16], :, tokens % 16]              # [n, hkv, d]
        out.append(w * rows[1:].sum(0) / (1 + w * (len(tokens) - 1)))
    return np.stack(out)


def check(got, want, n, bits, out_type, weight_type):
    rel = 2 * (n / 16 + 64) * 2.0 ** -24 + 2.0 ** -17 + HALF_STEP[weight_type]
    if weight_type == "f16":
        rel += 2.0 ** (-25 - LIFT + bits)
    limit = (HALF_STEP[out_type] + rel) * (1 + 2.0 ** -7) * want + (2.0 ** -25 if out_type == "f16" else 0)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= limit).all(), f"worst {np.max(err / want):.2e} of the value, allowed {np.min(limit / want):.2e}"


def decode_batch(dev, hq, hkv, d, window, sinks):
    """Enough work that a warp has hundreds of blocks in a row: 96 sequences of
    8000 tokens that share 512 blocks (nothing is written)."""
    lens = np.full(96, 8000, dtype=np.int32)
    lens[5], lens[90] = 7003, 17
    tables = np.tile(np.arange(512, dtype=np.int32), (96, 1))
    seen = []
    for n in lens:
        t = np.arange(n)
        seen.append(t[(t < sinks) | (t >= n - window)] if window else t)
    q = torch.zeros((96, hq, d), device=dev)
    q[:, :, 0] = 1
    return lens, tables, seen, q


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (7000, 1)])
def test_decode_16_bit_cache(gpu, dtype, head_dim, bits, window, sinks):
    k, v = cache(512, 8, head_dim, 3)
    lens, tables, seen, q = decode_batch(gpu, 16, 8, head_dim, window, sinks)
    kc, vc = (torch.from_numpy(x).to(gpu, TORCH_DTYPES[dtype]) for x in (k, v))
    bt, cl = to_dev(gpu, tables, lens)
    out = pa.paged_attention_decode_window(q.to(TORCH_DTYPES[dtype]), kc, vc, bt, cl, window, sinks,
                                           scale_for(bits))
    pa.check_status()
    want = expected(v, tables, seen, bits).repeat(2, axis=1)
    check(out, want, 8000, bits, dtype, dtype)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (7000, 1)])
def test_decode_8_bit_cache(gpu, dtype, head_dim, bits, window, sinks):
    k, v = cache(512, 8, head_dim, 5)
    lens, tables, seen, q = decode_batch(gpu, 16, 8, head_dim, window, sinks)
    codes = [torch.from_numpy(oq.encode(x * s)).to(gpu).view(torch.float8_e4m3fn)
             for x, s in ((k, 4), (v, 0.5))]
    scales = [torch.full((512, 8), s, device=gpu) for s in (0.25, 2.0)]
    bt, cl = to_dev(gpu, tables, lens)
    out = pa.paged_attention_decode_q8(q.to(TORCH_DTYPES[dtype]), *codes, *scales, bt, cl, window, sinks,
                                       scale_for(bits))
    pa.check_status()
    want = expected(v, tables, seen, bits).repeat(2, axis=1)
    check(out, want, 8000, bits, dtype, "f16")
