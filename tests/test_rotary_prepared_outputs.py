"""A prepared call without a tensor for what it computes is refused: nobody
could read it (CPU only)."""

import pytest
import torch

import pagedattention_decode_attention_gb300 as pa


def test_refused():
    rot = pa.Rotary(64, "cpu")
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    c16 = torch.zeros(2, 4, 16, 64, dtype=torch.bfloat16)
    c8, s = c16.to(torch.float8_e4m3fn), torch.ones(2, 4)
    pos = torch.zeros(2, dtype=torch.int32)
    bt, cl, qs = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    slots, ws = torch.zeros(2, dtype=torch.int64), torch.empty(256, dtype=torch.uint8)
    for name, call in (
            ("q_out", lambda: pa.prepare_rotary(q, None, pos, rot, None, None)),
            ("q_out", lambda: pa.prepare_rotary(q, q, pos, rot, None, q)),
            ("k_out", lambda: pa.prepare_rotary(q, q, pos, rot, q, None)),
            ("q_out", lambda: pa.prepare_rotary_kv_append(q, q, q, pos, rot, c16, c16, slots, None)),
            ("q_out", lambda: pa.prepare_rotary_kv_append_q8(q, q, q, None, rot, c8, c8, s, s, bt, cl, qs, None)),
            ("out", lambda: pa.prepare_decode_rotary_append_run(q, q, q, None, rot, slots, c16, c16, bt, cl, 0.1, ws,
                                                                None)),
            ("out", lambda: pa.prepare_decode_q8_rotary_append_run(q, q, q, None, rot, c8, c8, s, s, bt, cl, 0, 0,
                                                                   0.1, ws, None))):
        with pytest.raises(ValueError, match=rf"\b{name} must be given"):
            call()
