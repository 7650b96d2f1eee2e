"""Calls given a stream of their own: the memory they allocate for themselves
(workspace, output) must not pass to other work while that stream still uses
it.  Nothing is launched where the ownership alone is looked at."""

import contextlib

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from pagedattention_decode_attention_gb300 import capi, ops
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.test_gpu_window import to_dev
from tests.window_helpers import cache16, cache8, window_tables

pytestmark = pytest.mark.gpu

LENS, NEW = [900, 30, 333], [5, 1, 40]


def case(dev):
    gen = np.random.default_rng(3)
    tables, nb = window_tables(LENS, LENS, 0, 0, gen)
    kc, vc = cache16(nb, 8, 128, "bf16", 5, dev)
    _, _, codes, scales = cache8(nb, 8, 128, 7, dev)
    bt, cl, qs = to_dev(dev, tables, LENS, np.concatenate([[0], np.cumsum(NEW)]))
    q = wl.normal((3, 32, 128), torch.bfloat16, 9, dev)
    rows = wl.normal((sum(NEW), 32, 128), torch.bfloat16, 10, dev)
    starts, blocks = to_dev(dev, [0, 3], [0])
    return {
        "decode_window": lambda **kw: pa.paged_attention_decode_window(q, kc, vc, bt, cl, 200, 4, 0.1, **kw),
        "decode_q8": lambda **kw: pa.paged_attention_decode_q8(q, *codes, *scales, bt, cl, 200, 4, 0.1, **kw),
        "prefill_window": lambda **kw: pa.paged_attention_prefill_window(rows, kc, vc, bt, cl, qs, 200, 4, 0.1,
                                                                         **kw),
        "decode": lambda **kw: pa.paged_attention_decode(q, kc, vc, bt, cl, 0.1, **kw),
        "prefill": lambda **kw: pa.paged_attention_prefill(rows, kc, vc, bt, cl, qs, 0.1, **kw),
        "shared_prefix": lambda **kw: pa.paged_attention_decode_shared_prefix(q, kc, vc, bt, cl, 0, 0.1, **kw),
        "grouped_prefix": lambda **kw: pa.paged_attention_decode_grouped_prefix(q, kc, vc, bt, cl, starts,
                                                                                blocks, 0.1, **kw),
    }


NAMES = ["decode_window", "decode_q8", "prefill_window", "decode", "prefill", "shared_prefix",
         "grouped_prefix"]


class Recorder:
    """The library with its launching entry points replaced by notes of the
    pointers they were given (sizes are still asked of the library itself)."""

    def __init__(self, lib):
        self._lib, self.pointers = lib, set()

    def __getattr__(self, name):
        if name.endswith("_size"):
            return getattr(self._lib, name)

        def note(*args):
            for a in args:
                a = getattr(a, "value", a)
                if isinstance(a, int) and a > 1 << 24:
                    self.pointers.add(a)
            return 0
        return note


@contextlib.contextmanager
def recorded(monkeypatch):
    fake = Recorder(capi.lib())
    with monkeypatch.context() as m:
        m.setattr(ops.capi, "lib", lambda: fake)
        yield fake


@pytest.mark.parametrize("name", NAMES)
def test_the_workspace_stays_with_its_stream(gpu, monkeypatch, name):
    """A workspace (and an output) that a call with ``stream=`` allocated and
    let go of is not what the next allocation on the current stream gets."""
    call = case(gpu)[name]
    side = torch.cuda.Stream(gpu)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with recorded(monkeypatch) as lib:
        before = torch.cuda.memory_stats(gpu)["allocation.all.allocated"]
        call(stream=side)
        made = torch.cuda.memory_stats(gpu)["allocation.all.allocated"] - before
    assert made == 2                                    # output and workspace
    # as many pieces of any size as could hold either: none of them may be one
    # of the addresses the launch was given
    new = [torch.empty(n, dtype=torch.uint8, device=gpu)
           for n in (512, 8192, 1 << 16, 1 << 18, 1 << 20, 3 << 20, 6 << 20, 12 << 20, 24 << 20, 48 << 20, 96 << 20)
           for _ in range(6)]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in new]
    live = set()
    for p in lib.pointers:
        if any(a <= p < b for a, b in spans):
            live.add(p)
    assert not live, "memory still in use on the call's stream was handed out again"


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_its_own(gpu, name):
    """The call on another stream, with memory of its own and the caller's
    stream at work beside it, gives what it gives on the current one."""
    call = case(gpu)[name]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream(gpu)
    junk = []
    for _ in range(10):
        side.wait_stream(torch.cuda.current_stream(gpu))
        out = call(stream=side)
        junk = [torch.full((n,), 0xA5, dtype=torch.uint8, device=gpu) for n in (1 << 16, 1 << 20, 8 << 20)]
        torch.cuda.current_stream(gpu).wait_stream(side)
        assert torch.equal(out, want)
    pa.check_status()
    assert len(junk) == 3
