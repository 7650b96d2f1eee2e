"""Pins of the rotary oracle, and the host side of the rotation against it (CPU
only)."""

import math

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from oracle import rotary as orot


@pytest.mark.parametrize("interleaved", [False, True])
def test_a_quarter_turn_by_hand(interleaved):
    """One pair, one position: (a, b) at w = pi / 2 becomes (-b, a)."""
    x = np.arange(1.0, 17.0).reshape(1, 1, 16)
    w = np.zeros(4)
    w[1] = math.pi / 2
    got, _ = orot.rotate(x, [1], w, interleaved)
    want = x.copy()
    a, b = (2, 3) if interleaved else (1, 5)
    want[0, 0, a], want[0, 0, b] = -x[0, 0, b], x[0, 0, a]
    np.testing.assert_allclose(got, want, atol=1e-14)


@pytest.mark.parametrize("interleaved", [False, True])
def test_is_a_rotation_matrix_power(interleaved):
    """Position p is the p-th power of position 1's matrix, its transpose the
    inverse, and products of two rows depend on the distance only."""
    gen = np.random.default_rng(1)
    w = orot.frequencies(16, 100.0)
    eye = np.eye(32)[:, None]
    one = orot.rotate(eye, [1] * 32, w, interleaved)[0][:, 0].T
    five = orot.rotate(eye, [5] * 32, w, interleaved)[0][:, 0].T
    back = orot.rotate(eye, [-5] * 32, w, interleaved)[0][:, 0].T
    np.testing.assert_allclose(np.linalg.matrix_power(one, 5), five, atol=1e-12)
    np.testing.assert_allclose(back, five.T, atol=1e-12)
    np.testing.assert_allclose(five @ back, np.eye(32), atol=1e-12)
    q, k = gen.standard_normal((2, 1, 1, 32))
    dots = [float((orot.rotate(q, [p + 7], w, interleaved)[0] * orot.rotate(k, [p], w, interleaved)[0]).sum())
            for p in (0, 3, 1000)]
    np.testing.assert_allclose(dots, dots[0], atol=1e-11)


CASES = [dict(base=10000.0), dict(base=500000.0), dict(base=10000.0, scaling="linear", factor=4.0),
         dict(base=10000.0, scaling="base", factor=8.0),
         dict(base=500000.0, scaling="bands", factor=8.0, original_context=8192, low=1.0, high=4.0),
         dict(base=10000.0, scaling="bands", factor=3.5, original_context=2048, low=1.0, high=32.0)]


@pytest.mark.parametrize("rotary_dim", [16, 48, 64, 112, 128])
@pytest.mark.parametrize("case", CASES, ids=lambda c: c.get("scaling", "plain"))
def test_frequencies(rotary_dim, case):
    got = pa.rotary_frequencies(rotary_dim, **case).numpy()
    # exp, log and pow of doubles: a few half steps each, of exponents up to 13
    np.testing.assert_allclose(got, orot.frequencies(rotary_dim, **case), rtol=2.0 ** -48)


def test_bands_keep_fast_pairs_and_stretch_slow_ones():
    plain = pa.rotary_frequencies(128, 10000.0)
    bands = pa.rotary_frequencies(128, 10000.0, "bands", 4.0, 4096, 1.0, 32.0)
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(bands[turns >= 32], plain[turns >= 32]) and (turns >= 32).any()
    slow = turns <= 1
    assert torch.allclose(bands[slow], plain[slow] / 4, rtol=1e-15, atol=0) and slow.any()
    assert (bands[1:] < bands[:-1]).all()


def test_turns():
    w = torch.tensor([0.0, math.pi, math.pi / 2, -math.pi / 2, 2 * math.pi, 1.0, -1.0, 1e-9, 12345.678])
    got = pa.rotary_turns(w.double())
    exact = [round((float(x) / (2 * math.pi) % 1.0) * 2 ** 64) % 2 ** 64 for x in w.double()]
    for g, e, x in zip(got.tolist(), exact, w.tolist()):
        # the division by a turn and the whole turns' subtraction, in 64 bits
        off = ((g - e + 2 ** 63) % 2 ** 64) - 2 ** 63
        assert abs(off) <= (abs(x) + 1) * 2.0 ** 64 * 2.0 ** -51, (x, g, e)
    assert got[0] == 0 and abs(got[1].item()) >= 2 ** 62
    assert pa.rotary_turns(torch.empty(0)).numel() == 0


def test_turns_of_far_positions():
    """position * turns wraps where the angle does: exact integers against the
    angle in long arithmetic."""
    w = orot.frequencies(128, 10000.0)
    t = pa.rotary_turns(torch.from_numpy(w)).numpy().astype(object)
    for p in (1, -1, 99991, 2 ** 31 - 1, -2 ** 31):
        frac = np.array([int(p) * int(x) % 2 ** 64 for x in t], dtype=float) / 2.0 ** 64
        want = (p * w / (2 * math.pi)) % 1.0
        off = np.abs((frac - want + 0.5) % 1.0 - 0.5)
        assert off.max() <= abs(p) * w.max() * 2.0 ** -50 + 2.0 ** -30


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=24), dict(rotary_dim=144),
                                dict(base=0.0), dict(base=float("nan")), dict(base=float("inf")),
                                dict(scaling="linear", factor=0.0), dict(scaling="base", factor=-1.0),
                                dict(scaling="bands", factor=2.0), dict(scaling="bands", factor=2.0,
                                                                        original_context=10, low=4.0, high=4.0)])
def test_frequencies_refuse(kw):
    kw = {"rotary_dim": 64, **kw}
    with pytest.raises(pa.PagedAttnError):
        pa.rotary_frequencies(**kw)


def test_rotary_refuses():
    with pytest.raises(ValueError):
        pa.rotary_frequencies(64, scaling="unheard of")
    for kw in (dict(head_dim=96), dict(head_dim=64, rotary_dim=72), dict(head_dim=64, rotary_dim=8),
               dict(head_dim=64, rotary_dim=80), dict(head_dim=64, magnitude=float("inf")),
               dict(head_dim=64, magnitude=float("nan")), dict(head_dim=64, frequencies=[1.0] * 31)):
        with pytest.raises(ValueError):
            pa.Rotary(device="cpu", **kw)
    with pytest.raises(pa.PagedAttnError):
        pa.Rotary(64, "cpu", frequencies=[float("nan")] * 32)


def test_rotary_keeps_what_it_was_given():
    r = pa.Rotary(64, "cpu", rotary_dim=32, frequencies=[0.5] * 16, interleaved=True, magnitude=1.25)
    assert (r.rotary_dim, r.interleaved, r.magnitude) == (32, True, 1.25)
    assert torch.equal(r.turns, pa.rotary_turns(torch.full((16,), 0.5)))
    t = r.transposed()
    assert torch.equal(t.turns, -r.turns) and (t.magnitude, t.interleaved) == (1.25, True)
    assert torch.equal(t.transposed().turns, r.turns)
