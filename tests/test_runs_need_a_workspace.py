"""The runs over a plan made earlier refuse to go without the workspace that
holds it (CPU only)."""

import pytest
import torch

import pagedattention_decode_attention_gb300 as pa

Q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
C16 = torch.zeros(2, 4, 16, 64, dtype=torch.bfloat16)
C8 = C16.to(torch.float8_e4m3fn)
S = torch.ones(2, 4)
BT, CL = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
QS = torch.tensor([0, 1], dtype=torch.int32)

CALLS = {
    "window_run": lambda: pa.paged_attention_decode_window_run(Q, C16, C16, BT, CL, 4, 1, 0.1, None),
    "window_prepare": lambda: pa.prepare_decode_window_run(Q, C16, C16, BT, CL, 4, 1, 0.1, None, Q),
    "q8_run": lambda: pa.paged_attention_decode_q8_run(Q, C8, C8, S, S, BT, CL, 0, 0, 0.1, None),
    "q8_prepare": lambda: pa.prepare_decode_q8_run(Q, C8, C8, S, S, BT, CL, 0, 0, 0.1, None, Q),
    "q8_append_run": lambda: pa.paged_attention_decode_q8_append_run(Q, Q, Q, C8, C8, S, S, BT, CL, 0, 0,
                                                                     0.1, None),
    "q8_append_prepare": lambda: pa.prepare_decode_q8_append_run(Q, Q, Q, C8, C8, S, S, BT, CL, 0, 0, 0.1,
                                                                 None, Q),
    "prefill_run": lambda: pa.paged_attention_prefill_window_run(Q, C16, C16, BT, CL, QS, 4, 1, 0.1, None),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_run_without_its_workspace_is_refused(name):
    with pytest.raises(ValueError, match="workspace"):
        CALLS[name]()
