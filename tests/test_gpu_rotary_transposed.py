"""The transposed rotation made within the call that uses it, as a backward pass
does: on another stream behind other work, and while a graph is captured."""

import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.rotary_helpers import rotary_of, same_bits

pytestmark = pytest.mark.gpu


def test_made_within_a_call_on_another_stream(gpu):
    """Its frequencies stand while the side stream still has to read them,
    whatever is allocated and written on the current one meanwhile."""
    rot, _ = rotary_of(pa, 128, gpu)
    g = wl.normal((64, 8, 128), torch.float32, 3, gpu)
    pos = torch.arange(64, dtype=torch.int32, device=gpu)
    out = torch.zeros_like(g)
    busy = torch.ones((4096, 4096), device=gpu)
    side, main = torch.cuda.Stream(gpu), torch.cuda.current_stream(gpu)
    kept = rot.transposed()
    want, _ = pa.rotary(g, None, pos, kept)

    def work(n):
        x = busy
        for _ in range(n):
            x = torch.mm(x, busy)
        return x

    def write():        # the frequencies' size and its neighbours
        return [torch.full((n,), 5, dtype=torch.int64, device=gpu) for n in (64, 128, 32, 16) for _ in range(50)]

    with torch.cuda.stream(side):       # (a kernel's first launch may wait for the whole device)
        work(2)
    write()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):       # some 80 ms
        work(40)
    pa.rotary(g, None, pos, rot.transposed(), q_out=out, stream=side)
    over = write()
    main.wait_stream(side)
    assert same_bits(out, want) and len(over) == 200


def test_made_while_a_graph_is_captured(gpu):
    rot, _ = rotary_of(pa, 64, gpu, interleaved=True)
    g = wl.normal((20, 4, 64), torch.bfloat16, 4, gpu)
    pos = torch.arange(20, dtype=torch.int32, device=gpu)
    out = torch.zeros_like(g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.rotary(g, None, pos, rot.transposed(), q_out=out)
    over = [torch.zeros(32, dtype=torch.int64, device=gpu) for _ in range(100)]
    for shift in (0, 77):
        pos += shift
        graph.replay()
        assert same_bits(out, pa.rotary(g, None, pos, rot.transposed())[0]) and len(over) == 100
    pa.check_status()
