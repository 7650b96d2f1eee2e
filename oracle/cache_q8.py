"""Oracle of the 8-bit cache: e4m3 codes with a power-of-two scale for each
(block, KV head), K and V apart.

TEST INFRASTRUCTURE ONLY: plain numpy, float64, from the definitions: the 256
code values from sign, exponent and mantissa, rounding by nearest value with
ties to the even code, the scale by trying exponents in turn.
"""

from __future__ import annotations

import numpy as np

BLOCK_SIZE = 16
EXP_MIN, EXP_MAX = -100, 120
CODE_MAX = 448.0


def code_values() -> np.ndarray:
    """Value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3
    mantissa bits; exponent 0 is subnormal, 0x7f / 0xff are NaN."""
    out = np.empty(256)
    for code in range(256):
        sign, e, m = -1.0 if code & 0x80 else 1.0, (code >> 3) & 15, code & 7
        if e == 15 and m == 7:
            out[code] = np.nan
        elif e == 0:
            out[code] = sign * m * 2.0 ** -9
        else:
            out[code] = sign * (1 + m / 8) * 2.0 ** (e - 7)
    return out


VALUES = code_values()
_POSITIVE = VALUES[:0x7F]                # codes 0 .. 0x7e, increasing


def encode(x: np.ndarray) -> np.ndarray:
    """Nearest code (uint8): ties to the even code, beyond +-448 the largest,
    NaN to 0x7f; the sign of zero is kept."""
    x = np.asarray(x, dtype=np.float64)
    size = np.minimum(np.abs(x), CODE_MAX)
    size = np.where(np.isnan(x), 0.0, size)
    above = np.clip(np.searchsorted(_POSITIVE, size, side="left"), 0, 0x7E)
    below = np.maximum(above - 1, 0)
    up, down = _POSITIVE[above] - size, size - _POSITIVE[below]
    code = np.where((up < down) | ((up == down) & (above % 2 == 0)), above, below)
    code = np.where(_POSITIVE[above] == size, above, code).astype(np.uint8)
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def decode(codes: np.ndarray) -> np.ndarray:
    return VALUES[codes]


def scale_for(x: np.ndarray) -> float:
    """The smallest power of two (exponent -100 .. 120) whose 448-fold holds
    every finite value of ``x``."""
    finite = np.abs(x[np.isfinite(x)])
    peak = float(finite.max()) if finite.size else 0.0
    for e in range(EXP_MIN, EXP_MAX + 1):
        if peak <= CODE_MAX * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** EXP_MAX


def kv_append_q8(k, v, k_codes, v_codes, k_scale, v_scale, block_tables, context_lens,
                 query_start) -> None:
    """In place: ``k`` / ``v`` ``[T, Hkv, d]`` (float), codes uint8 ``[NB, Hkv,
    16, d]``, scales ``[NB, Hkv]``.  Sequence ``b``'s rows ``query_start[b] ..``
    are its newest tokens."""
    for b in range(len(context_lens)):
        first, last = int(query_start[b]), int(query_start[b + 1])
        ctx = int(context_lens[b])
        begin = ctx - (last - first)
        if last == first:
            continue
        for blk in range(begin // BLOCK_SIZE, (ctx - 1) // BLOCK_SIZE + 1):
            lo = max(begin, blk * BLOCK_SIZE)
            hi = min(ctx, (blk + 1) * BLOCK_SIZE)
            phys = int(block_tables[b][blk])
            held = lo - blk * BLOCK_SIZE         # older tokens in the block
            for rows, codes, scales in ((k, k_codes, k_scale), (v, v_codes, v_scale)):
                for h in range(rows.shape[1]):
                    new = rows[first + lo - begin: first + hi - begin, h].astype(np.float64)
                    s = scale_for(new)
                    if held:
                        s = max(s, float(scales[phys, h]))
                        if s > scales[phys, h]:
                            old = decode(codes[phys, h, :held]) * float(scales[phys, h])
                            codes[phys, h, :held] = encode(old / s)
                    codes[phys, h, held: held + hi - lo] = encode(new / s)
                    scales[phys, h] = s


def block_dequantize(codes, scales, pairs, out) -> None:
    """``out[dst] = scale * code`` of block ``src`` for every pair, in order."""
    for src, dst in pairs:
        out[int(dst)] = decode(codes[int(src)]) * np.asarray(scales[int(src)],
                                                            dtype=np.float64)[:, None, None]
