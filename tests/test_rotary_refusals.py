"""Calls the rotary entry points refuse on the host, before any launch (CPU
only)."""

import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from pagedattention_decode_attention_gb300 import build, capi

ROT = dict(turns=256, rdim=64, inter=0, mag=1.0)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.lib()


def refused(lib, name, base, kw):
    a = dict(base)
    assert set(kw) <= set(a)
    a.update(kw)
    rc = getattr(lib, name)(*a.values())
    assert rc == 0 or lib.pa_last_error()
    return rc


ROWS = dict(q=256, k=256, pos=256, **ROT, n=3, hq=8, hkv=2, d=128, qs=1024, ks=256, qos=1024, kos=256,
            dtype=2, qo=512, ko=512, stream=None)
APPEND = dict(q=256, k=256, v=256, pos=256, **ROT, kc=256, vc=256, slots=256, n=3, hq=8, hkv=2, d=128,
              nb=8, qs=1024, ks=256, vs=256, qos=1024, dtype=2, qo=512, stream=None)
APPEND8 = dict(q=256, k=256, v=256, pos=None, **ROT, kc=256, vc=256, ksc=256, vsc=256, bt=256, cl=256,
               qstart=256, b=2, n=3, hq=8, hkv=2, d=128, mb=4, nb=8, qs=1024, ks=256, vs=256, qos=1024,
               dtype=2, qo=512, stream=None)
DECODE = dict(q=256, k=256, v=256, pos=None, **ROT, slots=256, kc=256, vc=256, bt=256, cl=256, b=2, hq=8,
              hkv=2, d=128, mb=4, nb=8, qs=1024, ks=256, vs=256, scale=0.1, dtype=2, out=512, ws=256,
              bytes=1 << 30, stream=None)
DECODE8 = dict(q=256, k=256, v=256, pos=None, **ROT, kc=256, vc=256, ksc=256, vsc=256, bt=256, cl=256,
               window=8, sinks=2, b=2, hq=8, hkv=2, d=128, mb=4, nb=8, qs=1024, ks=256, vs=256, scale=0.1,
               dtype=2, out=512, ws=256, bytes=1 << 30, stream=None)
ALL = {"pa_rotary": ROWS, "pa_rotary_kv_append": APPEND, "pa_rotary_kv_append_q8": APPEND8,
       "pa_paged_attention_decode_rotary_append_run": DECODE,
       "pa_paged_attention_decode_q8_rotary_append_run": DECODE8}


@pytest.mark.parametrize("name", sorted(ALL))
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), 2), (dict(d=96, rdim=96), 2), (dict(turns=None), 1), (dict(turns=260), 1),
    (dict(rdim=0), 1), (dict(rdim=8), 1), (dict(rdim=40), 1), (dict(rdim=144), 1), (dict(inter=2), 1),
    (dict(mag=float("nan")), 1), (dict(mag=float("inf")), 1), (dict(q=None), 1), (dict(k=None), 1),
    (dict(q=264), 1), (dict(k=264), 1), (dict(qs=-1024), 1), (dict(ks=4), 1), (dict(qs=1020), 1),
    (dict(ks=1 << 41), 1),
])
def test_every_call_refuses(lib, name, kw, status):
    assert refused(lib, name, ALL[name], kw) == status


@pytest.mark.parametrize("name,kw,status", [
    ("pa_rotary", dict(pos=None), 1), ("pa_rotary", dict(n=-1), 1), ("pa_rotary", dict(hq=-1), 1),
    ("pa_rotary", dict(hq=0, hkv=0), 1), ("pa_rotary", dict(hq=1 << 17), 1), ("pa_rotary", dict(qo=None), 1),
    ("pa_rotary", dict(ko=None), 1), ("pa_rotary", dict(ko=520), 1), ("pa_rotary", dict(qos=1016), 1),
    ("pa_rotary", dict(kos=0), 1),
    ("pa_rotary_kv_append", dict(pos=None), 1), ("pa_rotary_kv_append", dict(v=None), 1),
    ("pa_rotary_kv_append", dict(v=264), 1), ("pa_rotary_kv_append", dict(vs=4), 1),
    ("pa_rotary_kv_append", dict(slots=None), 1), ("pa_rotary_kv_append", dict(kc=None), 1),
    ("pa_rotary_kv_append", dict(vc=264), 1), ("pa_rotary_kv_append", dict(nb=0), 1),
    ("pa_rotary_kv_append", dict(hkv=0), 1), ("pa_rotary_kv_append", dict(n=-1), 1),
    ("pa_rotary_kv_append", dict(qo=None), 1), ("pa_rotary_kv_append", dict(qos=512), 1),
    ("pa_rotary_kv_append_q8", dict(v=None), 1), ("pa_rotary_kv_append_q8", dict(vsc=None), 1),
    ("pa_rotary_kv_append_q8", dict(bt=None), 1), ("pa_rotary_kv_append_q8", dict(cl=None), 1),
    ("pa_rotary_kv_append_q8", dict(qstart=None), 1), ("pa_rotary_kv_append_q8", dict(b=-1), 1),
    ("pa_rotary_kv_append_q8", dict(mb=0), 1), ("pa_rotary_kv_append_q8", dict(mb=1 << 28), 1),
    ("pa_rotary_kv_append_q8", dict(b=1 << 30), 1), ("pa_rotary_kv_append_q8", dict(qo=None), 1),
    ("pa_rotary_kv_append_q8", dict(hq=-1), 1), ("pa_rotary_kv_append_q8", dict(vc=264), 1),
    ("pa_paged_attention_decode_rotary_append_run", dict(v=None), 1),
    ("pa_paged_attention_decode_rotary_append_run", dict(v=264), 1),
    ("pa_paged_attention_decode_rotary_append_run", dict(vs=-8), 1),
    ("pa_paged_attention_decode_rotary_append_run", dict(slots=None), 1),
    ("pa_paged_attention_decode_rotary_append_run", dict(out=None), 1),
    ("pa_paged_attention_decode_rotary_append_run", dict(bt=None), 1),
    ("pa_paged_attention_decode_rotary_append_run", dict(ws=None), 1),
    ("pa_paged_attention_decode_rotary_append_run", dict(bytes=64), 1),
    ("pa_paged_attention_decode_rotary_append_run", dict(hq=9), 1),
    ("pa_paged_attention_decode_rotary_append_run", dict(hq=18), 2),
    ("pa_paged_attention_decode_q8_rotary_append_run", dict(v=None), 1),
    ("pa_paged_attention_decode_q8_rotary_append_run", dict(v=264), 1),
    ("pa_paged_attention_decode_q8_rotary_append_run", dict(dtype=0), 2),
    ("pa_paged_attention_decode_q8_rotary_append_run", dict(window=-1), 1),
    ("pa_paged_attention_decode_q8_rotary_append_run", dict(ksc=None), 1),
    ("pa_paged_attention_decode_q8_rotary_append_run", dict(ws=264), 1),
    ("pa_paged_attention_decode_q8_rotary_append_run", dict(bytes=64), 1),
    ("pa_paged_attention_decode_q8_rotary_append_run", dict(hq=18), 2),
])
def test_a_call_refuses(lib, name, kw, status):
    assert refused(lib, name, ALL[name], kw) == status


@pytest.mark.parametrize("name", sorted(ALL))
def test_empty_calls_are_noops(lib, name):
    a = dict(ALL[name])
    for key in a:
        if isinstance(a[key], int) and a[key] in (256, 512) and key not in ("ks", "vs", "kos"):
            a[key] = None
    if "b" in a:
        a["b"] = 0
    else:
        a["n"] = 0
    assert getattr(lib, name)(*a.values()) == 0


def test_python_binding_refuses():
    rot = pa.Rotary(64, "cpu")
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    c16 = torch.zeros(2, 4, 16, 64, dtype=torch.bfloat16)
    c8, s = c16.to(torch.float8_e4m3fn), torch.ones(2, 4)
    pos = torch.zeros(2, dtype=torch.int32)
    bt, cl, qs = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    slots, ws = torch.zeros(2, dtype=torch.int64), torch.empty(256, dtype=torch.uint8)
    for call in (lambda: pa.rotary(q, q, pos, rot),
                 lambda: pa.rotary(None, None, pos, rot),
                 lambda: pa.rotary_kv_append(q, q, q, pos, rot, c16, c16, slots),
                 lambda: pa.rotary_kv_append_q8(q, q, q, None, rot, c8, c8, s, s, bt, cl, qs),
                 lambda: pa.paged_attention_decode_rotary_append_run(q, q, q, None, rot, slots, c16, c16,
                                                                     bt, cl, 0.1, ws),
                 lambda: pa.paged_attention_decode_q8_rotary_append_run(q, q, q, None, rot, c8, c8, s, s,
                                                                        bt, cl, 0, 0, 0.1, ws)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: pa.paged_attention_decode_rotary_append_run(q, q, q, None, rot, slots, c16, c16,
                                                                     bt, cl, 0.1, None),
                 lambda: pa.prepare_decode_q8_rotary_append_run(q, q, q, None, rot, c8, c8, s, s, bt, cl,
                                                                0, 0, 0.1, None, q)):
        with pytest.raises(ValueError, match="workspace"):
            call()


def test_the_rotating_decode_gives_up_by_whole_warps():
    """Its lanes hand query columns to one another for every block, so a wait
    that runs out is voted on (read in the source: the path cannot be staged)."""
    import os
    import re
    with open(os.path.join(build.PKG, "csrc", "decode.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    kernel = text[text.index("decode_kernel(const __grid_constant__"):text.index("decode_f32_kernel")]
    rows = r"arrived = mbar_wait_bounded\(my_q,[^;]*;\s*if constexpr \(ROT != 0\) arrived = __all_sync\(0xffffffffu, arrived\);"
    blocks = r"if constexpr \(ROT != 0\) \{\s*if \(!__all_sync\(0xffffffffu, dev::mbar_try_wait\([^;]*&&\s*" \
             r"!__all_sync\(0xffffffffu, mbar_wait_bounded\("
    assert len(re.findall(rows, kernel)) == 1 and len(re.findall(blocks, kernel)) == 1
