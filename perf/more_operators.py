"""Measured cases of the rotary position operators.

A row x of a head (query or key) of the token at position p is rotated in its
first ``rdim`` columns: pair i of them turns by the angle p * w_i and is
multiplied by a magnitude,

    (a, b) -> m * (a cos - b sin, b cos + a sin),

where the pairs are columns (i, i + rdim / 2), or (2i, 2i + 1) where they are
interleaved; the other columns pass through.  Five kinds of pass:

* ``rotary``      the query and key rows of a batch of tokens, read from where a
  fused projection left them; ``transposed`` turns the other way, which takes
  the gradients of the rotated rows to those of the rows;
* ``append``      a layer's step over new tokens: queries rotated, keys rotated
  into their slots of a paged cache (blocks of 16 tokens), values beside them;
* ``append_q8``   the same into a cache of 8 bits (e4m3 codes with a power-of-two
  scale for each block and KV head);
* ``decode``      one decode step: each sequence's new key rotated and stored
  with its value, and its rotated query's attention over the whole cache;
* ``decode_q8``   that over the 8-bit cache, optionally with a sliding window and
  a few first tokens that stay visible.

``run`` computes them in elementary torch operations where ``own`` is false and
by the library's calls where it is true; both return the same tensors.  A
rotated query is not rounded before the decode kinds' attention; a key is held
in the cache's type, and that is what attention reads.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 16
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EXP_MIN, EXP_MAX = -100, 120      # exponents a block's scale may have
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def _case(name, kind, dtype, heads, kv_heads, dim, batch, lo, hi, new_lo=1, new_hi=1, **more):
    c = dict(name=name, kind=kind, dtype=dtype, heads=heads, kv_heads=kv_heads, dim=dim,
             batch=batch, lo=lo, hi=hi, new_lo=new_lo, new_hi=new_hi, rdim=dim, base=10000.0,
             interleaved=False, scaling="none", factor=1.0, original=0, low=0.0, high=0.0,
             magnitude=1.0, transposed=False, window=0, sinks=0, mix=0)
    c.update(more)
    return c


LONG = dict(base=500000.0, scaling="bands", factor=8.0, original=8192, low=1.0, high=4.0)


def listed():
    cases = [
        # the newest token of a single chat
        _case("rotary_one", "rotary", "bf16", 32, 8, 128, 1, 101, 101),
        # a batch of prompt chunks at ragged positions of a stretched context
        _case("rotary_prompts", "rotary", "bf16", 32, 8, 128, 16, 2000, 65536, 200, 2048, **LONG),
        # back through a layer in 32 bits: interleaved pairs in half of each head
        _case("rotary_grad", "rotary", "f32", 32, 32, 64, 5, 300, 2047, 300, 2047, rdim=32,
              interleaved=True, transposed=True),
        # a decode step's new tokens, ahead of a cascade or windowed decode
        _case("append_step", "append", "bf16", 32, 8, 128, 128, 128, 8192),
        # the 8B-shaped workload's prompt chunks, some of them shorter
        _case("append_prompts", "append", "bf16", 32, 8, 128, 16, 528, 8704, 301, 512),
        # many short prompts, a KV head for every query head, interleaved in part of the head
        _case("append_mha", "append", "f16", 32, 32, 64, 33, 7, 500, 7, 500, rdim=32,
              interleaved=True),
        # a decode step's new tokens into 8 bits
        _case("append_q8_step", "append_q8", "bf16", 32, 8, 128, 128, 128, 8192),
        # prompt chunks of uneven length into 8 bits
        _case("append_q8_prompts", "append_q8", "bf16", 32, 8, 128, 16, 300, 8192, 200, 2048),
        # one chat turn just begun
        _case("decode_one", "decode", "bf16", 32, 8, 128, 1, 101, 101),
        # the 7B-shaped serving batch: a KV head for every query head
        _case("decode_mha", "decode", "f16", 32, 32, 128, 64, 16, 2048),
        # the 8B-shaped serving batch over 8 bits, grouped heads, ragged lengths
        _case("decode_q8_gqa", "decode_q8", "bf16", 32, 8, 128, 128, 128, 8192, base=500000.0),
        # long conversations with a window, interleaved in part of the head; blocks behind the
        # window have been freed
        _case("decode_q8_window", "decode_q8", "bf16", 32, 4, 64, 19, 1000, 65536, rdim=32,
              interleaved=True, scaling="linear", factor=4.0, window=4000, sinks=4),
    ]
    return [dict(c, mix=i + 1) for i, c in enumerate(cases)]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["rotary", "rotary", "append", "append", "append_q8", "decode", "decode",
                       "decode_q8"])
    heads, kv = rng.choice([(32, 8), (32, 8), (32, 32), (32, 4), (20, 4)])
    dim = rng.choice([128, 128, 64])
    types = ["bf16", "f16", "f32"] if kind in ("rotary", "append") else ["bf16", "f16"]
    c = _case("x", kind, rng.choice(types), heads, kv, dim, 1, 1, 1, mix=rng.randrange(1 << 20))
    del c["name"]
    c["rdim"] = rng.choice([dim, dim, dim // 2, dim // 4, dim - 16])
    c["interleaved"] = rng.random() < 0.4
    c["base"] = rng.choice([10000.0, 500000.0, 1000000.0])
    how = rng.choice(["none", "none", "linear", "base", "bands"])
    if how != "none":
        c.update(scaling=how, factor=rng.choice([2.0, 4.0, 8.0, 3.5]))
        if how == "bands":
            low, high = rng.choice([(1.0, 4.0), (1.0, 32.0)])
            c.update(original=rng.choice([2048, 4096, 8192]), low=low, high=high,
                     magnitude=rng.choice([1.0, 0.1 * math.log(c["factor"]) + 1.0]))
    c["transposed"] = kind == "rotary" and rng.random() < 0.4
    if kind.startswith("decode"):
        c["hi"] = _log_int(rng, 64, 32768)
        c["lo"] = _log_int(rng, 1, c["hi"])
        c["batch"] = _log_int(rng, 1, max(1, min(128, (1 << 27) // (c["hi"] * kv * dim))))
        if kind == "decode_q8" and rng.random() < 0.4:
            c["window"] = _log_int(rng, 100, 4096)
            c["sinks"] = rng.choice([0, 1, 4, 16])
    else:
        c["new_hi"] = rng.choice([1, _log_int(rng, 2, 2048)])
        c["new_lo"] = _log_int(rng, 1, c["new_hi"])
        c["hi"] = _log_int(rng, c["new_hi"], max(65536 if kind == "rotary" else 8192, c["new_hi"]))
        c["lo"] = _log_int(rng, c["new_lo"], c["hi"])
        most = (1 << 25) // (c["new_hi"] * (heads + 2 * kv) * dim) if c["new_hi"] > 1 else 128
        if kind != "rotary":
            most = min(most, (1 << 27) // (c["hi"] * kv * dim))
        c["batch"] = _log_int(rng, 1, max(1, min(128, most)))
    return c


# ---------------------------------------------------------------- lengths
def _lengths(case):
    """(context lengths, new tokens) of the case's sequences, spread over the
    logarithm; the new tokens are a sequence's last."""
    g = np.random.default_rng(9000 + case["mix"])
    b = case["batch"]

    def spread(lo, hi):
        x = np.rint(np.exp(g.uniform(math.log(lo), math.log(hi + 0.49), b)))
        return np.clip(x, lo, hi).astype(np.int64)

    ctx = spread(case["lo"], case["hi"])
    ctx[: b // 32] = case["hi"]
    return ctx, np.minimum(spread(case["new_lo"], case["new_hi"]), ctx)


def _visible(case, ctx):
    """Tokens of each sequence that its last query sees."""
    if not case["window"]:
        return ctx
    first = np.minimum(case["sinks"], np.maximum(ctx - case["window"], 0))
    return np.minimum(ctx, case["window"]) + first


def work(case):
    ctx, new = _lengths(case)
    hq, hkv, d, r = case["heads"], case["kv_heads"], case["dim"], case["rdim"]
    size = {"f32": 4, "f16": 2, "bf16": 2}[case["dtype"]]
    t = int(new.sum())
    kind = case["kind"]
    turns = 3.0 * t * (hq + hkv) * r                  # four products and two sums a pair
    small = 4 * t + 8 * (r // 2)                      # positions, frequencies
    if kind == "rotary":
        return {"bytes": 2 * size * t * (hq + hkv) * d + small, "flops": turns}
    if kind == "append":
        return {"bytes": 2 * size * t * (hq + 2 * hkv) * d + small + 8 * t, "flops": turns}
    blocks = int(((ctx - 1) // BLOCK - (ctx - new) // BLOCK + 1).sum())
    if kind == "append_q8":
        # queries read and written, keys and values read, their codes written;
        # a block that begins earlier has its scales read, every one has them
        # written
        return {"bytes": 2 * size * t * hq * d + 2 * t * hkv * d * (size + 1) + small
                + 4 * 2 * hkv * (blocks + int(((ctx - new) % BLOCK > 0).sum())) + 4 * blocks
                + 8 * len(ctx), "flops": turns + 4.0 * t * hkv * d}
    seen = int(_visible(case, ctx).sum())
    elem = 1 if kind == "decode_q8" else size
    scales = 8 * hkv * (seen // BLOCK) if elem == 1 else 0
    # the cache's visible tokens but the new ones, which are read from the new
    # rows and stored
    return {"bytes": 2 * (seen - t) * hkv * d * elem + scales + 2 * t * hkv * d * (size + elem)
            + 2 * size * t * hq * d + 4 * (seen // BLOCK + 2 * t) + 8 * (r // 2),
            "flops": turns + 4.0 * seen * hq * d}


# ----------------------------------------------------------------- inputs
def _block_exponent(peak):
    """Smallest e with peak <= 448 * 2^e (peak: largest finite magnitude)."""
    m, x = torch.frexp(peak.double())
    e = torch.where(m <= 0.875, x - 9, x - 8)
    e = torch.where(peak > 0, e, torch.full_like(e, EXP_MIN))
    return e.clamp(EXP_MIN, EXP_MAX)


def _quantise(rows, scale):
    """e4m3 codes of rows / scale (a power of two: the division is exact)."""
    return (rows / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def prepare(case, seed):
    dev = torch.device("cuda")
    ctx, new = _lengths(case)
    hq, hkv, d, dt = case["heads"], case["kv_heads"], case["dim"], TYPES[case["dtype"]]
    kind, w, s = case["kind"], case["window"], case["sinks"]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    host = np.random.default_rng([seed, case["mix"]])
    b, total = len(ctx), int(new.sum())
    starts = np.concatenate([[0], np.cumsum(new)])
    st = dict(case=case, scale=1.0 / math.sqrt(d), max_ctx=int(ctx.max()))

    # what a layer's projection wrote: a token's queries, keys and values side
    # by side; channels of uneven size
    def rows(n, heads):
        x = torch.randn((n, heads, d), generator=g, device=dev)
        return x * torch.exp(0.5 * torch.randn((1, heads, d), generator=g, device=dev))

    if case["transposed"]:
        # gradients, each a tensor of its own
        st["q"], st["k"] = rows(total, hq).to(dt), rows(total, hkv).to(dt)
    else:
        qkv = rows(total, hq + 2 * hkv).to(dt)
        st["q"], st["k"], st["v"] = qkv.split([hq, hkv, hkv], dim=1)
    position = np.concatenate([np.arange(c - n, c) for c, n in zip(ctx, new)])
    st["positions"] = torch.from_numpy(position.astype(np.int32)).to(dev)
    st["q_out"] = torch.empty((total, hq, d), dtype=dt, device=dev)
    st["frequencies"] = _frequencies(case).to(dev)

    if kind == "rotary":
        st["k_out"] = torch.empty((total, hkv, d), dtype=dt, device=dev)
    else:
        # a shuffled pool; blocks no query sees have been freed (-1).  A pass
        # that reads no older tokens has a pool of the blocks it writes to and
        # a few others
        nblk = (ctx + BLOCK - 1) // BLOCK
        mb = int(nblk.max())
        col = np.arange(mb)[None, :]
        held = col < nblk[:, None]
        if kind.startswith("append"):
            held &= col >= ((ctx - new) // BLOCK)[:, None]
        if w:
            low = np.maximum(ctx - w, 0)[:, None]
            held &= (col * BLOCK < s) | ((col + 1) * BLOCK > low)
        count = int(held.sum())
        nb = count + max(2, count // 10)
        tables = np.full((b, mb), -1, dtype=np.int32)
        tables[held] = host.permutation(nb)[:count].astype(np.int32)
        st["block_tables"] = torch.from_numpy(tables).to(dev)
        st["context_lens"] = torch.from_numpy(ctx.astype(np.int32)).to(dev)
        st["query_start"] = torch.from_numpy(starts.astype(np.int32)).to(dev)
        seq = np.repeat(np.arange(b), new)
        slots = tables[seq, position // BLOCK].astype(np.int64) * BLOCK + position % BLOCK
        st["slots"] = torch.from_numpy(slots).to(dev)
        st["touched"] = torch.from_numpy(np.unique(slots // BLOCK)).to(dev)
        for name, flat in (("k", True), ("v", False)):
            x = torch.randn((nb, hkv, BLOCK, d), generator=g, device=dev)
            # keys with channels of uneven size, values with tokens of uneven size
            x *= torch.exp(0.5 * torch.randn((1, hkv, 1, d) if flat else (nb, hkv, BLOCK, 1),
                                             generator=g, device=dev))
            if kind.endswith("q8"):
                e = _block_exponent(x.abs().amax(dim=(2, 3)))
                scale = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
                st[name + "_cache"] = _quantise(x, scale[:, :, None, None])
                st[name + "_scale"] = scale.contiguous()
            else:
                st[name + "_cache"] = x.to(dt)
            del x

    # what a serving loop keeps: the rotation's frequencies, over the layers of
    # a step the workspace with its plan, and the calls bound to their buffers
    if own:
        import pagedattention_decode_attention_gb300 as pa
        scaling = None if case["scaling"] == "none" else case["scaling"]
        rot = pa.Rotary(d, dev, rotary_dim=case["rdim"], base=case["base"],
                        interleaved=case["interleaved"], scaling=scaling, factor=case["factor"],
                        original_context=case["original"], low=case["low"], high=case["high"],
                        magnitude=case["magnitude"])
        cache = [st[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale") if n in st]
        if kind == "rotary":
            st["op"] = pa.prepare_rotary(st["q"], st["k"], st["positions"],
                                         rot.transposed() if case["transposed"] else rot,
                                         st["q_out"], st["k_out"])
        elif kind == "append":
            st["op"] = pa.prepare_rotary_kv_append(st["q"], st["k"], st["v"], st["positions"], rot,
                                                   *cache, st["slots"], st["q_out"])
        elif kind == "append_q8":
            st["op"] = pa.prepare_rotary_kv_append_q8(
                st["q"], st["k"], st["v"], None, rot, *cache, st["block_tables"],
                st["context_lens"], st["query_start"], st["q_out"])
        elif kind == "decode":
            ws = pa.alloc_workspace(b, hq, hkv, d, mb, dev)
            pa.paged_attention_decode_plan(st["context_lens"], hq, hkv, d, mb, ws)
            st["op"] = pa.prepare_decode_rotary_append_run(
                st["q"], st["k"], st["v"], None, rot, st["slots"], *cache, st["block_tables"],
                st["context_lens"], st["scale"], ws, st["q_out"])
        else:
            ws = pa.alloc_window_workspace(b, hq, hkv, d, mb, dev)
            pa.paged_attention_decode_window_plan(st["context_lens"], w, s, hq, hkv, d, mb, ws)
            st["op"] = pa.prepare_decode_q8_rotary_append_run(
                st["q"], st["k"], st["v"], None, rot, *cache, st["block_tables"],
                st["context_lens"], w, s, st["scale"], ws, st["q_out"])
    return st


# ------------------------------------------------------------ plain forms
def _frequencies(case):
    """Angle per position of each pair, in 64 bits."""
    r = case["rdim"]
    base, factor = case["base"], case["factor"]
    if case["scaling"] == "base":
        base = base * factor ** (r / (r - 2))
    w = base ** -(torch.arange(0, r, 2, dtype=torch.float64) / r)
    if case["scaling"] == "linear":
        w = w / factor
    if case["scaling"] == "bands":
        turns = case["original"] * w / (2 * math.pi)
        keep = ((turns - case["low"]) / (case["high"] - case["low"])).clamp(0.0, 1.0)
        w = w * (keep + (1 - keep) / factor)
    return w


def _rotate(st, x):
    """Rows [T, H, d] rotated, in 32 bits (the angles in 64)."""
    case, r = st["case"], st["case"]["rdim"]
    angle = st["positions"].double()[:, None] * st["frequencies"]
    c = (case["magnitude"] * angle.cos()).float()[:, None]
    s = (case["magnitude"] * angle.sin()).float()[:, None]
    if case["transposed"]:
        s = -s
    y = x.float()
    if case["interleaved"]:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = y[..., : r // 2], y[..., r // 2: r]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, y[..., r:]], -1)


def _place(cache, rows, slots):
    cache[slots // BLOCK, :, slots % BLOCK] = rows.to(cache.dtype)


def _place_q8(cache, scale, x, slots, touched):
    """Writes the rows of ``x`` (32 bits) into the 8-bit blocks they belong to:
    a block's scale holds its largest new row, and grows where it has older
    tokens, whose codes are then rounded anew."""
    blocks, unit, older = touched
    fresh = ~older[:, 0]
    codes = cache.view(torch.uint8)
    off = slots % BLOCK
    peak = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    most = torch.zeros((blocks.numel(), x.shape[1]), device=x.device)
    most.scatter_reduce_(0, unit[:, None].expand_as(peak), peak, "amax")
    want = torch.ldexp(torch.ones_like(most), _block_exponent(most))
    old = scale[blocks]
    grown = torch.where(fresh[:, None], want, torch.maximum(old, want))
    held = codes[blocks]
    moved = held.view(torch.float8_e4m3fn).float() * (old / grown)[..., None, None]
    moved = moved.to(torch.float8_e4m3fn).view(torch.uint8)
    held = torch.where(older[:, None, :, None] & (grown > old)[..., None, None], moved, held)
    held[unit, :, off] = _quantise(x, grown[unit][..., None]).view(torch.uint8)
    codes[blocks] = held
    scale[blocks] = grown


def _touched(st):
    """The blocks that the new tokens go to, which of them each token's is, and
    which of their slots hold older tokens (those in front of the new)."""
    blocks, slots = st["touched"], st["slots"]
    place = torch.zeros(st["k_cache"].shape[0], dtype=torch.long, device=slots.device)
    place[blocks] = torch.arange(blocks.numel(), device=slots.device)
    unit = place[slots // BLOCK]
    first = torch.full_like(blocks, BLOCK).scatter_reduce_(0, unit, slots % BLOCK, "amin")
    return blocks, unit, torch.arange(BLOCK, device=slots.device)[None] < first[:, None]


def _gather(cache, scale, phys, off):
    """Rows [B, n, Hkv, D] in 32 bits of the tokens at (phys, off)."""
    if scale is None:
        return cache[phys, :, off].float()
    rows = cache.view(torch.uint8)[phys, :, off].view(torch.float8_e4m3fn).float()
    return rows * scale[phys][..., None]


def _attend(st, q):
    """Decode attention of the rows q (32 bits) over the cache as it is now."""
    case = st["case"]
    ctx, tables = st["context_lens"].long(), st["block_tables"].long()
    b, hq, d = q.shape
    hkv, w, s, dev = case["kv_heads"], case["window"], case["sinks"], q.device
    if w:
        # the first tokens, then the window's, each token once
        n = min(w, st["max_ctx"])
        last = ctx[:, None] - n + torch.arange(n, device=dev)
        first = torch.arange(s, device=dev).expand(b, s)
        at = torch.cat([first, last], 1)
        ok = torch.cat([first < (ctx[:, None] - w).clamp(min=0), last >= 0], 1)
    else:
        at = torch.arange(st["max_ctx"], device=dev).expand(b, -1)
        ok = at < ctx[:, None]
    at = torch.where(ok, at, 0)
    phys = torch.where(ok, torch.gather(tables, 1, at // BLOCK), 0)
    off = at % BLOCK
    k = _gather(st["k_cache"], st.get("k_scale"), phys, off)
    scores = torch.einsum("bhgd,bnhd->bhgn", q.view(b, hkv, hq // hkv, d), k) * st["scale"]
    del k
    scores = scores.masked_fill(~ok[:, None, None], float("-inf"))
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    v = _gather(st["v_cache"], st.get("v_scale"), phys, off)
    return torch.einsum("bhgn,bnhd->bhgd", p, v).reshape(b, hq, d)


def _answer(st, out):
    """A pass's outputs: what it returns and every buffer it changes."""
    names = [n for n in ("k_cache", "v_cache", "k_scale", "v_scale") if n in st]
    return {"out": out, **{n: st[n] for n in names}}


def run(state):
    kind = state["case"]["kind"]
    if own:
        state["op"]()
        if kind == "rotary":
            return {"q": state["q_out"], "k": state["k_out"]}
        return _answer(state, state["q_out"])
    q, k = _rotate(state, state["q"]), _rotate(state, state["k"])
    dt = state["q"].dtype
    if kind == "rotary":
        return {"q": q.to(dt), "k": k.to(dt)}
    if kind.endswith("q8"):
        touched = _touched(state)
        _place_q8(state["k_cache"], state["k_scale"], k, state["slots"], touched)
        _place_q8(state["v_cache"], state["v_scale"], state["v"].float(), state["slots"], touched)
    else:
        _place(state["k_cache"], k, state["slots"])
        _place(state["v_cache"], state["v"], state["slots"])
    if kind.startswith("decode"):
        q = _attend(state, q)
    return _answer(state, q.to(dt))


# ------------------------------------------------------------------ exact
def _e4m3_nearest(x):
    """x rounded to the nearest e4m3 value (ties to even), in 64 bits."""
    size = x.abs()
    e = torch.frexp(size)[1] - 1
    step = torch.ldexp(torch.ones_like(x), e.clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _turned(case, x, positions):
    """Rows rotated as complex numbers in 64 bits."""
    r, half = case["rdim"], case["rdim"] // 2
    w = []
    for i in range(half):
        log_base = math.log(case["base"])
        if case["scaling"] == "base":
            log_base += math.log(case["factor"]) * r / (r - 2)
        f = math.exp(-2.0 * i / r * log_base)
        if case["scaling"] == "linear":
            f /= case["factor"]
        if case["scaling"] == "bands":
            n = case["original"] * f / (2 * math.pi)
            if n < case["low"]:
                f /= case["factor"]
            elif n < case["high"]:
                part = (n - case["low"]) / (case["high"] - case["low"])
                f = (1 - part) * f / case["factor"] + part * f
        w.append(-f if case["transposed"] else f)
    w = torch.tensor(w, dtype=torch.float64, device=x.device)
    angle = torch.outer(positions.double(), w)
    turn = torch.polar(torch.full_like(angle, case["magnitude"]), angle)[:, None]
    y = x.double().clone()
    if case["interleaved"]:
        y[..., :r] = torch.view_as_real(torch.view_as_complex(
            y[..., :r].reshape(*y.shape[:2], half, 2).contiguous()) * turn).flatten(-2)
    else:
        z = torch.complex(y[..., :half].contiguous(), y[..., half:r].contiguous()) * turn
        y[..., :half], y[..., half:r] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    ctx, new = _lengths(case)
    kind = case["kind"]
    q, k = (_turned(case, st[n], st["positions"]) for n in ("q", "k"))
    if kind == "rotary":
        return {"q": q, "k": k}
    dt, dev, hkv = st["q"].dtype, q.device, case["kv_heads"]
    phys, off = st["slots"] // BLOCK, st["slots"] % BLOCK
    held, seen = {}, {}              # outputs, and the values attention reads
    if kind.endswith("q8"):
        for name, x in (("k", k), ("v", st["v"].double())):
            codes = st[name + "_cache"].view(torch.uint8).view(torch.float8_e4m3fn).double()
            scale = st[name + "_scale"].double()
            for b, (n, t) in enumerate(zip(ctx.tolist(), new.tolist())):
                row = int(st["query_start"][b])
                # the chunk's own blocks, one after the other
                at = n - t
                while at < n:
                    end = min(n, (at // BLOCK + 1) * BLOCK)
                    p, lo = int(phys[row]), at % BLOCK
                    new_rows = x[row: row + end - at].transpose(0, 1)
                    peak = new_rows.abs().amax((1, 2))
                    # the smallest power of two whose 448-fold holds the peak
                    e = torch.floor(torch.log2(peak.clamp(min=1e-300) / 448.0)) - 1
                    for _ in range(3):
                        e = torch.where(peak > 448.0 * torch.exp2(e), e + 1, e)
                    s = torch.exp2(e.clamp(EXP_MIN, EXP_MAX))
                    if lo:
                        s = torch.maximum(s, scale[p])
                        codes[p, :, :lo] = _e4m3_nearest(codes[p, :, :lo] * (scale[p] / s)[:, None, None])
                    codes[p, :, lo: lo + end - at] = _e4m3_nearest(new_rows / s[:, None, None])
                    scale[p] = s
                    row, at = row + end - at, end
            held[name + "_cache"], held[name + "_scale"] = codes, scale
            seen[name] = codes * scale[:, :, None, None]
    else:
        for name, x in (("k", k), ("v", st["v"].double())):
            cache = st[name + "_cache"].double()
            cache[phys, :, off] = x
            held[name + "_cache"] = cache
            # (attention reads what the cache's type holds)
            seen[name] = cache.clone()
            seen[name][phys, :, off] = x.to(dt).double()
    if kind.startswith("append"):
        return {"out": q, **held}
    w, s, group = case["window"], case["sinks"], case["heads"] // hkv
    out = torch.empty_like(q)
    for b in range(len(ctx)):
        n = int(ctx[b])
        low = max(n - w, 0) if w else 0
        at = np.concatenate([np.arange(min(s, low)), np.arange(low, n)])
        block = torch.from_numpy(st["block_tables"][b].cpu().numpy().astype(np.int64)[at // BLOCK]).to(dev)
        slot = torch.from_numpy(at % BLOCK).to(dev)
        keys, values = (seen[c][block, :, slot].transpose(0, 1) for c in ("k", "v"))
        x = torch.einsum("hgd,hnd->hgn", q[b].view(hkv, group, -1), keys) * st["scale"]
        out[b] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), values).reshape(case["heads"], -1)
    return {"out": out, **held}
