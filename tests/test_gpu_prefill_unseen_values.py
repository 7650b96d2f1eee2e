"""Windowed chunked prefill over caches with infinities and NaN among the
values: a row's output depends on the tokens it sees and on nothing else, also
where other rows of its chunk see more or less than it does."""

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from oracle import windowed as ow
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.gpu_helpers import TORCH_DTYPES, to_f32_numpy
from tests.test_gpu_window import to_dev
from tests.window_helpers import assert_within, bound, cache16, window_tables

pytestmark = pytest.mark.gpu


def run_case(dev, lens, new, hq, hkv, d, dtype, window, sinks, bad, rows, seed=11):
    """``bad``: (sequence, token, head, columns, value) to put into V; rows:
    checked against the oracle.  Returns how many checked rows see a bad
    value and how many do not."""
    gen = np.random.default_rng(seed)
    tables, nb = window_tables(lens, lens, 0, 0, gen)
    kc, vc = cache16(nb, hkv, d, dtype, seed, dev)
    for b, t, h, cols, x in bad:
        vc[int(tables[b, t // 16]), h, t % 16, cols] = x
    qs = np.concatenate([[0], np.cumsum(new)])
    q = wl.normal((int(qs[-1]), hq, d), TORCH_DTYPES[dtype], seed * 10 + 1, dev)
    lens = np.asarray(lens)
    bt, cl, st = to_dev(dev, tables, lens, qs)
    out = pa.paged_attention_prefill_window(q, kc, vc, bt, cl, st, window, sinks, d ** -0.5)
    pa.check_status()
    with np.errstate(invalid="ignore"):
        ref, spread, size = ow.prefill(to_f32_numpy(q), to_f32_numpy(kc), to_f32_numpy(vc), tables, lens,
                                       qs, window, sinks, d ** -0.5, rows=rows)
    got = out.float().cpu().numpy()[sorted(rows)]
    ref, spread, size = (x[sorted(rows)] for x in (ref, spread, size))
    odd = ~np.isfinite(ref)
    assert not np.isfinite(got[odd]).any(), "a row that sees the value has lost it"
    whole = ~odd.any(-1)
    keep = np.where(odd, np.nan, ref)                       # (assert_within passes over NaN)
    tokens = min(int(lens.max()), window + sinks) if window else int(lens.max())
    vmax = float(vc.float().nan_to_num(0, 0, 0).abs().max())
    limit = bound(np.where(odd, 0, ref), np.where(odd, 0, spread), size, tokens, dtype, dtype, vmax)
    assert_within(torch.from_numpy(got), keep, limit)
    return int((~whole).sum()), int(whole.sum())


BAD = [float("inf"), -float("inf"), float("nan")]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("heads", [(4, 4), (8, 2), (5, 1), (8, 1)], ids=["g1", "g4", "g5", "g8"])
def test_values_that_only_other_rows_see(gpu, dtype, head_dim, heads):
    """Bad values at tokens that early rows' windows hold and later ones have
    left, at tokens that only later rows see, and among the first tokens'
    neighbours; in one column or all, of one KV head."""
    hq, hkv = heads
    lens, new = [700, 200, 60], [300, 200, 60]
    bad = [(0, 345, 0, slice(None), BAD[0]), (0, 500, 0, slice(7, 8), BAD[1]), (0, 699, 0, slice(None), BAD[2]),
           (1, 5, 0, slice(3, 5), BAD[2]), (1, 120, 0, slice(0, 1), BAD[0]), (2, 59, 0, slice(None), BAD[1])]
    rows = set(range(0, 560, 9)) | {299, 298, 300, 301, 499, 500, 559, 558}
    seen, unseen = run_case(gpu, lens, new, hq, hkv, head_dim, dtype, 100, 4, bad, rows)
    assert seen > 0 and unseen > 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
def test_split_key_ranges(gpu, dtype, head_dim):
    """Few rows over a long window: the key range is split over CTAs, and a bad
    value lies in one part of it, seen by some rows and by others not."""
    lens, new = [5000], [40]
    bad = [(0, 4961 - 3000, 0, slice(None), BAD[2]), (0, 4990, 1, slice(2, 3), BAD[0])]
    seen, unseen = run_case(gpu, lens, new, 8, 2, head_dim, dtype, 3000, 16, bad, set(range(0, 40, 3)) | {39})
    assert seen > 0 and unseen > 0


@pytest.mark.parametrize("head_dim", [64, 128])
def test_first_tokens_and_no_window_left(gpu, head_dim):
    """A bad first token that every row sees, and one just past the first
    tokens that no row or only the first rows see."""
    lens, new = [300], [290]
    bad = [(0, 2, 0, slice(1, 2), BAD[0]), (0, 6, 1, slice(None), BAD[2])]
    seen, unseen = run_case(gpu, lens, new, 8, 2, head_dim, "bf16", 40, 5, bad, set(range(0, 290, 7)))
    assert seen > 0 and unseen > 0


@pytest.mark.parametrize("head_dim", [64, 128])
def test_every_value_bad(gpu, head_dim):
    """A cache of nothing but NaN ends (with NaN), and leaves the next call's
    results alone."""
    gen = np.random.default_rng(17)
    lens, new = np.array([900, 300]), np.array([260, 300])
    tables, nb = window_tables(lens, lens, 0, 0, gen)
    kc, vc = cache16(nb, 2, head_dim, "bf16", 17, gpu)
    qs = np.concatenate([[0], np.cumsum(new)])
    q = wl.normal((int(qs[-1]), 8, head_dim), torch.bfloat16, 171, gpu)
    bt, cl, st = to_dev(gpu, tables, lens, qs)
    ws = pa.alloc_prefill_workspace(2, int(qs[-1]), 8, 2, head_dim, gpu)
    args = (bt, cl, st, 200, 4, 0.1)
    want = pa.paged_attention_prefill_window(q, kc, vc, *args, workspace=ws)
    out = pa.paged_attention_prefill_window(q, kc, torch.full_like(vc, float("nan")), *args, workspace=ws)
    assert torch.isnan(out).all()
    out = pa.paged_attention_prefill_window(q, torch.full_like(kc, float("nan")), vc, *args, workspace=ws)
    assert torch.isnan(out).all()
    assert torch.equal(pa.paged_attention_prefill_window(q, kc, vc, *args, workspace=ws), want)
    pa.check_status()
