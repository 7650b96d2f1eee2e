"""Calls the sliding-window and 8-bit entry points refuse on the host, before
any launch (CPU only)."""

import ctypes as C

import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from pagedattention_decode_attention_gb300 import build, capi


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.lib()


def _decode(lib, q8=False, run=False, **kw):
    a = dict(q=256, k=256, v=256, ks=256, vs=256, bt=256, cl=256, window=8, sinks=2, num_seqs=2,
             hq=8, hkv=2, d=128, mb=4, nb=8, scale=0.125, dtype=2, out=256, ws=256, bytes=1 << 30)
    a.update(kw)
    name = "pa_paged_attention_decode_" + ("q8" if q8 else "window") + ("_run" if run else "")
    ptrs = [a["q"], a["k"], a["v"]] + ([a["ks"], a["vs"]] if q8 else []) + [a["bt"], a["cl"]]
    return getattr(lib, name)(*ptrs, a["window"], a["sinks"], a["num_seqs"], a["hq"], a["hkv"],
                              a["d"], a["mb"], a["nb"], a["scale"], a["dtype"], a["out"], a["ws"],
                              a["bytes"], None)


@pytest.mark.parametrize("run", [False, True])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(dtype=7), 2), (dict(d=96), 2),
    (dict(hq=9), 1), (dict(hq=18), 2), (dict(hkv=0), 1), (dict(mb=0), 1), (dict(nb=0), 1),
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(bt=None), 1),
    (dict(cl=None), 1), (dict(out=None), 1), (dict(q=264), 1), (dict(k=264), 1),
    (dict(out=264), 1), (dict(ws=None), 1), (dict(ws=264), 1), (dict(bytes=64), 1),
    (dict(num_seqs=-1), 1), (dict(num_seqs=1 << 20, mb=1 << 20), 1), (dict(mb=1 << 28), 1),
])
def test_decode_refuses(lib, q8, run, kw, status):
    assert _decode(lib, q8, run, **kw) == status
    assert lib.pa_last_error()


def test_q8_decode_refuses_what_only_it_has(lib):
    assert _decode(lib, True, dtype=0) == 2            # fp32 queries
    assert _decode(lib, True, ks=None) == 1
    assert _decode(lib, True, vs=None) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(window=-1), 1), (dict(dtype=0), 2), (dict(dtype=7), 2), (dict(d=96), 2), (dict(hq=18), 2),
    (dict(nb=0), 1), (dict(q=None), 1), (dict(kn=None), 1), (dict(vn=None), 1), (dict(kn=264), 1),
    (dict(vn=264), 1), (dict(vc=264), 1), (dict(ks=None), 1), (dict(ws=None), 1), (dict(bytes=64), 1),
])
def test_append_run_refuses(lib, kw, status):
    a = dict(q=256, kn=256, vn=256, kc=256, vc=256, ks=256, vs=256, bt=256, cl=256, window=8, sinks=2,
             num_seqs=2, hq=8, hkv=2, d=128, mb=4, nb=8, scale=0.125, dtype=2, out=256, ws=256,
             bytes=1 << 30, stream=None)
    a.update(kw)
    assert lib.pa_paged_attention_decode_q8_append_run(*a.values()) == status
    assert lib.pa_last_error()


def test_append_run_without_sequences(lib):
    assert lib.pa_paged_attention_decode_q8_append_run(
        *[None] * 9, 8, 2, 0, 8, 2, 128, 4, 8, 0.125, 2, None, None, 0, None) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(window=-1), 1), (dict(sinks=-2), 1), (dict(d=80), 2), (dict(cl=None), 1),
    (dict(ws=None), 1), (dict(bytes=8), 1), (dict(hq=7), 1),
])
def test_plan_refuses(lib, kw, status):
    a = dict(cl=256, window=8, sinks=2, num_seqs=2, hq=8, hkv=2, d=128, mb=4, ws=256, bytes=1 << 30)
    a.update(kw)
    assert lib.pa_paged_attention_decode_window_plan(
        a["cl"], a["window"], a["sinks"], a["num_seqs"], a["hq"], a["hkv"], a["d"], a["mb"],
        a["ws"], a["bytes"], None) == status


def test_workspace_size(lib):
    n = C.c_size_t(0)
    size = lib.pa_paged_attention_decode_window_workspace_size
    assert size(128, 32, 8, 128, 512, C.byref(n)) == 0 and n.value >= 128 * 4
    assert size(128, 32, 8, 128, 512, None) == 1
    assert size(1 << 20, 32, 8, 128, 1 << 20, C.byref(n)) == 1
    assert size(4, 32, 0, 128, 4, C.byref(n)) == 1
    assert size(4, 32, 8, 72, 4, C.byref(n)) == 2
    assert pa.paged_attention_decode_window_workspace_size(0, 32, 8, 128, 4) >= 0


@pytest.mark.parametrize("kw,status", [
    (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(dtype=5), 2), (dict(d=32), 2),
    (dict(hq=18), 2), (dict(q=None), 1), (dict(q=264), 1), (dict(qs=None), 1), (dict(bytes=8), 1),
])
def test_prefill_refuses(lib, kw, status):
    a = dict(q=256, k=256, v=256, bt=256, cl=256, qs=256, window=8, sinks=2, num_seqs=2, total_q=9,
             hq=8, hkv=2, d=128, mb=4, nb=8, scale=0.125, dtype=2, out=256, ws=256, bytes=1 << 30)
    a.update(kw)
    for name in ("pa_paged_attention_prefill_window", "pa_paged_attention_prefill_window_run"):
        assert getattr(lib, name)(
            a["q"], a["k"], a["v"], a["bt"], a["cl"], a["qs"], a["window"], a["sinks"],
            a["num_seqs"], a["total_q"], a["hq"], a["hkv"], a["d"], a["mb"], a["nb"], a["scale"],
            a["dtype"], a["out"], a["ws"], a["bytes"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=9), 2), (dict(d=96), 2), (dict(hkv=0), 1), (dict(nb=0), 1), (dict(k=None), 1),
    (dict(kc=None), 1), (dict(ks=None), 1), (dict(bt=None), 1), (dict(qs=None), 1),
    (dict(k=260), 1), (dict(vc=264), 1), (dict(tokens=-1), 1), (dict(mb=0), 1), (dict(mb=1 << 28), 1),
    (dict(num_seqs=1 << 30), 1),
])
def test_append_refuses(lib, kw, status):
    a = dict(k=256, v=256, kc=256, vc=256, ks=256, vs=256, bt=256, cl=256, qs=256, num_seqs=2,
             tokens=5, hkv=2, d=128, mb=4, nb=8, dtype=2)
    a.update(kw)
    assert lib.pa_kv_append_q8(a["k"], a["v"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["cl"],
                               a["qs"], a["num_seqs"], a["tokens"], a["hkv"], a["d"], a["mb"],
                               a["nb"], a["dtype"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=9), 2), (dict(d=96), 2), (dict(pairs=None), 1), (dict(ko=None), 1), (dict(n=-1), 1),
    (dict(nob=0), 1), (dict(ko=264), 1), (dict(kc=264), 1), (dict(ks=None), 1),
])
def test_dequantize_refuses(lib, kw, status):
    a = dict(kc=256, vc=256, ks=256, vs=256, pairs=256, n=3, hkv=2, d=128, nb=8, nob=8, dtype=2,
             ko=256, vo=256)
    a.update(kw)
    assert lib.pa_block_dequantize(a["kc"], a["vc"], a["ks"], a["vs"], a["pairs"], a["n"], a["hkv"],
                                   a["d"], a["nb"], a["nob"], a["dtype"], a["ko"], a["vo"],
                                   None) == status


def test_empty_calls_are_noops(lib):
    assert _decode(lib, num_seqs=0, q=None, k=None, ws=None, bytes=0) == 0
    assert _decode(lib, True, num_seqs=0, q=None, ks=None, ws=None, bytes=0) == 0
    assert lib.pa_kv_append_q8(*[None] * 9, 0, 0, 2, 128, 4, 8, 2, None) == 0
    assert lib.pa_kv_append_q8(*[None] * 9, 3, 0, 2, 128, 4, 8, 2, None) == 0
    assert lib.pa_block_dequantize(*[None] * 5, 0, 2, 128, 8, 8, 2, None, None, None) == 0


def test_python_binding_refuses_host_tensors():
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    c8 = torch.zeros(2, 4, 16, 64).to(torch.float8_e4m3fn)
    s = torch.ones(2, 4)
    bt, cl = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    qs = torch.tensor([0, 1], dtype=torch.int32)
    c16 = c8.to(torch.bfloat16)
    with pytest.raises(ValueError):
        pa.paged_attention_decode_q8(q, c8, c8, s, s, bt, cl, 0, 0, 0.1)
    with pytest.raises(ValueError):
        pa.paged_attention_decode_window(q, c16, c16, bt, cl, 4, 1, 0.1)
    with pytest.raises(ValueError):
        pa.paged_attention_prefill_window(q, c16, c16, bt, cl, qs, 4, 1, 0.1)
    with pytest.raises(ValueError):
        pa.kv_append_q8(q, q, c8, c8, s, s, bt, cl, qs)
    with pytest.raises(ValueError):
        pa.block_dequantize(c8, c8, s, s, torch.zeros(1, 2, dtype=torch.int64), c16, c16)


@pytest.mark.parametrize("window,sinks", [(1 << 32, 0), ((1 << 32) + 5, 0), (4, 1 << 31), (-(1 << 31) - 1, 0)])
def test_windows_past_32_bits_do_not_wrap(window, sinks):
    from pagedattention_decode_attention_gb300 import ops
    with pytest.raises(ValueError, match="32 bits"):
        ops._window_ints(window, sinks)
