"""Bounded device-side waits, read in the sources (CPU only).

A wait that runs out cannot be staged on a GPU without making it hang for the
while, so what must hold on that path is checked in the kernels' text."""

import os
import re

from pagedattention_decode_attention_gb300 import build

CSRC = os.path.join(build.PKG, "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_a_run_that_gave_up_voids_its_plan():
    """Counters of a run that gave up are not what the next one expects, so
    the plan's signature goes on that path in every planned kernel."""
    text = source("decode_window.cu")
    tail = text[text.index("if (!__syncthreads_and(ok))"):]
    assert re.match(r"if \(!__syncthreads_and\(ok\)\) \{[^}]*p\.header\[kHdrSignature\], 0\)[^}]*return;", tail)
    text = source("prefill.cu")
    assert re.search(r"void void_plan\(const Params& p\) \{\s*atomicExch\(&p\.header\[kHdrSignature\], 0\);", text)
    # the mma.sync kernel's way out, and the tcgen05 kernel's
    assert re.search(r"if \(!ok\) \{\s*if \(producer\) \{[^}]*void_plan\(p\);\s*\}\s*return;", text)
    assert re.search(r"if \([^)]*!all_ok\) void_plan\(p\);", text)


def test_a_voided_plan_does_not_part_a_running_block():
    """A thread block may start while another voids the plan: whether there is
    one is decided for whole warps (decode) or by the one thread that hands
    out the items (prefill)."""
    text = source("decode_window.cu")
    kernel = text[text.index("attend_kernel("):text.index("cudaError_t configure()")]
    assert re.search(r"planned = __all_sync\(0xffffffffu, hdr\.x == p\.signature\)", kernel)
    assert not re.search(r"if \(hdr\.x != p\.signature\)", kernel)
    text = source("prefill.cu")
    compared = re.findall(r"[^\n]*\bx (?:<|>=) total\b[^\n]*", text)
    assert len(compared) == 2 and all("kNoItem" in line for line in compared)


def statements(text, call):
    """(the statement up to the call, the lines before it, the text behind it)
    of every call."""
    for m in re.finditer(re.escape(call) + r"\(", text):
        start = max(text.rfind(c, 0, m.start()) for c in ";{}")
        yield text[start + 1:m.start()], text[:start + 1].splitlines()[-8:], text[m.end():m.end() + 300]


def test_warps_give_up_as_one():
    """A lane that gives up by itself leaves its warp's others at their next
    vote or shuffle for ever.  So a wait whose result is used either is voted
    on or belongs to a single lane."""
    single = re.compile(r"if \((?:lane == 0|producer|threadIdx\.x == 0)\b")
    seen = 0
    for name in ("prefill.cu", "decode_window.cu"):
        for before, above, behind in statements(source(name), "mbar_wait_bounded"):
            seen += 1
            alone = before.strip() in ("dev::", "") or re.fullmatch(r"\s*if \([^!]*\) dev::", before)
            voted = "__all_sync(" in before or \
                re.match(r"[^;]*ok = false;[^;]*(?:;[^;]*){0,5}\bok = __all_sync\(0xffffffffu, ok\);", behind)
            one = single.search(before) or any(single.search(line) for line in above)
            assert alone or voted or one, f"{name}: {before.strip()}"
    assert seen > 10
