"""The transposed rotation shares its rotation's frequencies (CPU only)."""

import pytest
import torch

import pagedattention_decode_attention_gb300 as pa


def test_it_is_made_once():
    r = pa.Rotary(64, "cpu", rotary_dim=32, base=500.0, interleaved=True, magnitude=1.5)
    t = r.transposed()
    assert r.transposed() is t and t.transposed() is r
    assert torch.equal(t.turns, -r.turns) and t.turns.is_contiguous()
    assert (t.rotary_dim, t.head_dim, t.interleaved, t.magnitude, t.device) == (32, 64, True, 1.5, r.device)


@pytest.mark.parametrize("keep", ["rotation", "transposed"])
def test_either_keeps_the_memory_of_both(keep):
    """One allocation, made with the rotation: a call on another stream or in a
    captured graph may make the transposed one on the way."""
    r = pa.Rotary(128, "cpu")
    t = r.transposed()
    assert r.turns.untyped_storage().data_ptr() == t.turns.untyped_storage().data_ptr()
    want = (r if keep == "rotation" else t).turns.clone()
    held = (r if keep == "rotation" else t).turns
    del r, t
    assert torch.equal(held, want)


def test_half_a_turn_is_its_own_opposite():
    import math
    r = pa.Rotary(64, "cpu", frequencies=[math.pi] * 16 + [-math.pi] * 16)
    both = (r.turns + r.transposed().turns).tolist()
    assert all(x in (0, -2 ** 63) for x in both)
