"""Oracle of attention with a sliding window and visible first tokens.

TEST INFRASTRUCTURE ONLY: plain numpy, float64.  A query at position ``p``
sees token ``t`` when ``t <= p`` and (``window == 0`` or ``t > p - window`` or
``t < num_sinks``); over the tokens it sees it is ordinary softmax attention.
Only visible tokens are gathered, one at a time, so table entries and slots
that nothing sees are never touched.
"""

from __future__ import annotations

import numpy as np

BLOCK_SIZE = 16


def visible_tokens(position: int, window: int, num_sinks: int) -> list[int]:
    """The tokens a query at ``position`` sees, in order."""
    return [t for t in range(position + 1)
            if window == 0 or t > position - window or t < num_sinks]


def gather_tokens(cache: np.ndarray, block_table, tokens, head: int,
                  scales: np.ndarray | None = None) -> np.ndarray:
    """Rows ``[len(tokens), d]`` (float64) of one KV head; ``scales``
    (``[num_blocks, num_kv_heads]``): what each block's values are multiplied by."""
    out = np.empty((len(tokens), cache.shape[3]), dtype=np.float64)
    for i, t in enumerate(tokens):
        physical = int(block_table[t // BLOCK_SIZE])
        assert 0 <= physical < cache.shape[0], "a visible token's block is in the pool"
        out[i] = cache[physical, head, t % BLOCK_SIZE].astype(np.float64)
        if scales is not None:
            out[i] *= float(scales[physical, head])
    return out


def attend(q: np.ndarray, keys: np.ndarray, values: np.ndarray, scale: float):
    """One query over the tokens it sees: ``(out, spread, size)`` with
    ``spread`` the weighted mean of ``|v|`` and ``size`` the largest
    ``scale * sum |q_d| |k_d|`` (what rounding errors are measured by)."""
    if keys.shape[0] == 0:
        zero = np.zeros(values.shape[1])
        return zero, zero, 0.0
    q = q.astype(np.float64)
    scores = scale * (keys @ q)
    weights = np.exp(scores - scores.max())
    weights /= weights.sum()
    size = abs(scale) * float((np.abs(keys) @ np.abs(q)).max())
    return weights @ values, weights @ np.abs(values), size


def prefill(q, k_cache, v_cache, block_tables, context_lens, query_start, window: int,
            num_sinks: int, scale: float, k_scale=None, v_scale=None, rows=None):
    """``(out, spread, size)`` for every query row and head: float64
    ``[total_q, Hq, d]`` twice and ``[total_q, Hq]``; rows of no sequence, and
    with ``rows`` the rows not in it, stay NaN."""
    total_q, num_q_heads, d = q.shape
    group = num_q_heads // k_cache.shape[1]
    out = np.full((total_q, num_q_heads, d), np.nan)
    spread = np.full((total_q, num_q_heads, d), np.nan)
    size = np.full((total_q, num_q_heads), np.nan)
    for b in range(len(context_lens)):
        first, last = int(query_start[b]), int(query_start[b + 1])
        for row in range(first, last):
            if rows is not None and row not in rows:
                continue
            position = int(context_lens[b]) - (last - first) + row - first
            tokens = visible_tokens(position, window, num_sinks)
            for g in range(k_cache.shape[1]):
                keys = gather_tokens(k_cache, block_tables[b], tokens, g, k_scale)
                values = gather_tokens(v_cache, block_tables[b], tokens, g, v_scale)
                for h in range(g * group, (g + 1) * group):
                    out[row, h], spread[row, h], size[row, h] = attend(q[row, h], keys, values, scale)
    return out, spread, size


def decode(q, k_cache, v_cache, block_tables, context_lens, window: int, num_sinks: int,
           scale: float, k_scale=None, v_scale=None, rows=None):
    """:func:`prefill` of one query per sequence, its newest token's; a
    sequence of no tokens gives zeros."""
    n = q.shape[0]
    some = [1 if int(c) > 0 else 0 for c in context_lens]
    starts = np.concatenate([[0], np.cumsum(some)])
    live = np.flatnonzero(some)
    wanted = None if rows is None else {int(starts[b]) for b in rows if some[b]}
    got = prefill(q[live], k_cache, v_cache, block_tables, context_lens, starts, window, num_sinks,
                  scale, k_scale, v_scale, wanted)
    full = []
    for part in got:
        x = np.zeros((n,) + part.shape[1:])
        x[live] = part
        full.append(x)
    return tuple(full)
