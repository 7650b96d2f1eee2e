"""Pins of the sliding-window and 8-bit cache oracles (CPU only)."""

import math

import numpy as np
import pytest
import torch

import oracle.attention as oa
from oracle import cache_q8 as oq
from oracle import windowed as ow
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.window_helpers import window_tables


def test_visible_tokens_by_hand():
    assert ow.visible_tokens(5, 0, 0) == [0, 1, 2, 3, 4, 5]
    assert ow.visible_tokens(5, 2, 0) == [4, 5]
    assert ow.visible_tokens(5, 2, 3) == [0, 1, 2, 4, 5]
    assert ow.visible_tokens(5, 2, 40) == [0, 1, 2, 3, 4, 5]
    assert ow.visible_tokens(5, 6, 0) == [0, 1, 2, 3, 4, 5]
    assert ow.visible_tokens(0, 1, 0) == [0]


def test_without_a_window_it_is_the_plain_oracle():
    gen = np.random.default_rng(3)
    lens = np.array([1, 17, 40, 0], dtype=np.int32)
    tables = wl.disjoint_tables(lens, 12, gen)
    q = gen.standard_normal((4, 4, 64))
    kc, vc = gen.standard_normal((2, 12, 2, 16, 64))
    ref = oa.paged_attention_decode(q, kc, vc, tables, lens, 0.125)
    for window in (0, 40, 1000):
        out, _, _ = ow.decode(q, kc, vc, tables, lens, window, 2, 0.125)
        np.testing.assert_allclose(out, ref, rtol=0, atol=1e-12)
    qs = np.array([0, 1, 5, 12, 12])
    q = gen.standard_normal((12, 4, 64))
    ref = oa.paged_attention_prefill(q, kc, vc, tables, lens, qs, 0.125)
    out, _, _ = ow.prefill(q, kc, vc, tables, lens, qs, 0, 7, 0.125)
    np.testing.assert_allclose(out, ref, rtol=0, atol=1e-12)


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 0), (5, 3), (16, 16), (30, 4)])
def test_windowed_prefill_is_masked_softmax(window, sinks):
    gen = np.random.default_rng(window * 7 + sinks)
    n = 45
    tables, nb = window_tables([n], [n], window, sinks, gen)
    kc, vc = gen.standard_normal((2, nb, 1, 16, 64))
    q = gen.standard_normal((n, 2, 64))
    out, _, _ = ow.prefill(q, kc, vc, tables, [n], [0, n], window, sinks, 0.125)
    k, v = (torch.from_numpy(oa.gather_sequence(c, tables[0], n)[:, 0]) for c in (kc, vc))
    i, j = torch.arange(n)[:, None], torch.arange(n)[None]
    seen = (j <= i) & ((i - j < window) | (j < sinks))
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).transpose(0, 1), k.expand(2, -1, -1), v.expand(2, -1, -1),
        attn_mask=seen, scale=0.125)
    np.testing.assert_allclose(out, want.transpose(0, 1).numpy(), rtol=0, atol=1e-12)


def test_freed_blocks_are_never_read():
    """Entries of blocks nothing sees are -1; the oracle asserts that it does
    not use them, and the first tokens' block stays."""
    gen = np.random.default_rng(11)
    tables, nb = window_tables([100, 33], [1, 3], 20, 4, gen)
    assert list(tables[0] >= 0) == [True, False, False, False, False, True, True]
    assert list(tables[1][:3] >= 0) == [True, True, True]
    kc, vc = gen.standard_normal((2, nb, 1, 16, 64))
    out, _, _ = ow.decode(gen.standard_normal((2, 1, 64)), kc, vc, tables, [100, 33], 20, 4, 0.1)
    assert np.isfinite(out).all()


def test_code_values():
    v = oq.VALUES
    assert v[0x7E] == 448.0 and v[0xFE] == -448.0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6
    assert v[0x38] == 1.0 and math.isnan(v[0x7F]) and math.isnan(v[0xFF])
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(v, t)


def test_encode_rounds_to_nearest_even():
    mid = (oq.VALUES[:0x7E] + oq.VALUES[1:0x7F]) / 2
    gen = np.random.default_rng(5)
    x = np.concatenate([mid, -mid, [0.0, -0.0, 448.0, 460.0, 1e9, -1e9, np.nan, 2.0 ** -11],
                        gen.standard_normal(20000) * np.exp(gen.uniform(-8, 7, 20000))])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = oq.encode(x)
    same = (got == want) | np.isnan(x)
    assert same.all()
    assert (got[np.isnan(x)] & 0x7F == 0x7F).all()
    assert oq.encode([np.inf])[0] == 0x7E and oq.encode([-np.inf])[0] == 0xFE


@pytest.mark.parametrize("peak,exponent", [(448.0, 0), (448.1, 1), (1.0, -8), (1.75, -8),
                                           (1.7500001, -7), (0.0, -100), (1e-38, -100),
                                           (3e38, 120), (896.0, 1)])
def test_scale_for(peak, exponent):
    x = np.array([peak / 3, -peak, np.inf, np.nan])
    assert oq.scale_for(x) == 2.0 ** exponent


def test_growing_a_scale_token_by_token():
    """Appending token by token ends at the scale of appending at once, and
    values that stay above the smallest step keep their codes' mantissas."""
    gen = np.random.default_rng(9)
    rows = gen.standard_normal((16, 1, 64)) * np.exp2(np.arange(16) % 5)[:, None, None]
    state = []
    for chunks in ([16], [1] * 16, [3, 5, 8]):
        codes = np.full((1, 1, 16, 64), 0x55, dtype=np.uint8)
        kv = [codes, codes.copy(), np.full((1, 1), 7.0), np.full((1, 1), 7.0)]
        at = 0
        for n in chunks:
            part = rows[at:at + n]
            at += n
            oq.kv_append_q8(part, 2 * part, kv[0], kv[1], kv[2], kv[3], np.zeros((1, 1), int), [at], [0, n])
        state.append(kv)
    for kv in state[1:]:
        assert kv[2] == state[0][2] and kv[3] == 2 * kv[2]
        a, b = oq.decode(kv[0]), oq.decode(state[0][0])
        normal = np.abs(b) >= 2.0 ** -6
        np.testing.assert_array_equal(a[normal], b[normal])
        assert np.abs(a - b).max() <= 2.0 ** -10 * 2      # two roundings under the smallest step
    x = np.abs(rows)
    err = np.abs(oq.decode(state[0][0])[0, 0] * state[0][2] - rows[:, 0])
    assert (err <= 2.0 ** -4 * x[:, 0] + 2.0 ** -10 * state[0][2]).all()


def test_append_leaves_the_rest_alone():
    codes = np.arange(3 * 16 * 64, dtype=np.int64).astype(np.uint8).reshape(3, 1, 16, 64) & 0x77
    k, v = codes.copy(), codes.copy()
    ks, vs = np.full((3, 1), 4.0), np.full((3, 1), 4.0)
    new = np.full((3, 1, 64), 2.0)
    oq.kv_append_q8(new, new, k, v, ks, vs, np.array([[2, 0]]), [18], [0, 3])
    np.testing.assert_array_equal(k[1], codes[1])
    np.testing.assert_array_equal(k[2, :, :15], codes[2, :, :15])    # 2.0 fits under scale 4
    np.testing.assert_array_equal(k[0, :, 2:], codes[0, :, 2:])      # behind the last token
    assert ks[2, 0] == 4.0 and ks[0, 0] == 2.0 ** -7
    np.testing.assert_array_equal(oq.decode(k[0, :, :2]) * ks[0, 0], np.full((1, 2, 64), 2.0))
