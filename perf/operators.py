"""Measured cases of the 8-bit cache and sliding-window operators.

Five kinds of pass over a paged K/V cache (blocks of 16 tokens, one block table
per sequence):

* ``decode_q8``      one decode step over a cache held in 8 bits (e4m3) with a
  power-of-two scale for each (block, KV head), optionally with a sliding
  window and a few first tokens that stay visible;
* ``decode_window``  one decode step over a 16-bit cache with a sliding window
  and first tokens;
* ``prefill_window`` causal chunked prefill with a sliding window and first
  tokens over a 16-bit cache;
* ``append_q8``      new tokens quantised into the 8-bit cache, then the blocks
  they touched read back as 16-bit values (what a prompt's next chunk attends
  over).

``run`` computes them in elementary torch operations where ``own`` is false and
by the library's calls where it is true; both return the same tensors.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 16
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
LOG2E = 1.4426950408889634
EXP_MIN, EXP_MAX = -100, 120      # exponents a block's scale may have
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one chat turn just begun: a single sequence, a hundred cached tokens
        dict(name="q8_one_short", kind="decode_q8", batch=1, lo=101, hi=101, heads=32, kv_heads=8,
             dim=128, dtype="bf16", window=0, sinks=0, mix=1),
        # the serving batch of the 8B-shaped workload, grouped heads, ragged lengths
        dict(name="q8_batch_gqa", kind="decode_q8", batch=128, lo=128, hi=8192, heads=32,
             kv_heads=8, dim=128, dtype="bf16", window=0, sinks=0, mix=2),
        # the 7B-shaped workload: a KV head for every query head
        dict(name="q8_batch_mha", kind="decode_q8", batch=64, lo=16, hi=2048, heads=32,
             kv_heads=32, dim=128, dtype="f16", window=0, sinks=0, mix=3),
        # long conversations with a window: blocks behind it have been freed
        dict(name="q8_window_long", kind="decode_q8", batch=19, lo=1000, hi=65536, heads=32,
             kv_heads=4, dim=64, dtype="bf16", window=4000, sinks=4, mix=4),
        # one very long stream, decoded token by token
        dict(name="window_one_long", kind="decode_window", batch=1, lo=100003, hi=100003,
             heads=32, kv_heads=8, dim=128, dtype="bf16", window=1024, sinks=4, mix=5),
        # a serving batch, some sequences still shorter than the window
        dict(name="window_batch", kind="decode_window", batch=64, lo=256, hi=32768, heads=32,
             kv_heads=8, dim=128, dtype="bf16", window=4096, sinks=64, mix=6),
        # odd window and first tokens, a KV head for every query head
        dict(name="window_mha_odd", kind="decode_window", batch=23, lo=1, hi=2047, heads=32,
             kv_heads=32, dim=64, dtype="f16", window=777, sinks=3, mix=7),
        # the last few tokens of one prompt
        dict(name="prefill_small", kind="prefill_window", batch=1, lo=700, hi=700, chunk_lo=37,
             chunk_hi=37, heads=4, kv_heads=4, dim=64, dtype="f16", window=250, sinks=4, mix=8),
        # a batch of prompt chunks at ragged positions
        dict(name="prefill_batch", kind="prefill_window", batch=16, lo=528, hi=8704, chunk_lo=512,
             chunk_hi=512, heads=32, kv_heads=8, dim=128, dtype="bf16", window=2048, sinks=4,
             mix=9),
        # two long prompts in large chunks of uneven length
        dict(name="prefill_long", kind="prefill_window", batch=2, lo=8000, hi=16384,
             chunk_lo=1500, chunk_hi=2048, heads=32, kv_heads=8, dim=128, dtype="bf16",
             window=4096, sinks=16, mix=10),
        # the new tokens of one decode step, a block each
        dict(name="append_step", kind="append_q8", batch=128, lo=128, hi=8192, chunk_lo=1,
             chunk_hi=1, heads=32, kv_heads=8, dim=128, dtype="bf16", window=0, sinks=0, mix=11),
        # prompt chunks of uneven length
        dict(name="append_prompts", kind="append_q8", batch=16, lo=300, hi=8192, chunk_lo=200,
             chunk_hi=2048, heads=32, kv_heads=8, dim=128, dtype="bf16", window=0, sinks=0,
             mix=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["decode_q8", "decode_q8", "decode_window", "decode_window",
                       "prefill_window", "append_q8"])
    heads, kv = rng.choice([(32, 8), (32, 8), (32, 32), (32, 4), (20, 4)])
    if kind == "prefill_window":
        heads, kv = rng.choice([(32, 8), (32, 8), (32, 4), (16, 16)])
    c = dict(kind=kind, heads=heads, kv_heads=kv, dim=rng.choice([128, 128, 64]),
             dtype=rng.choice(["bf16", "f16"]), mix=rng.randrange(1 << 20))
    if kind == "prefill_window":
        c["dim"] = 128
        c["chunk_hi"] = _log_int(rng, 17, 2048)
        c["chunk_lo"] = _log_int(rng, max(1, c["chunk_hi"] // 4), c["chunk_hi"])
        c["hi"] = _log_int(rng, c["chunk_hi"], 16384)
        c["lo"] = _log_int(rng, c["chunk_hi"], c["hi"])
        c["batch"] = _log_int(rng, 1, max(1, min(16, (64 << 20) // (c["chunk_hi"] * c["hi"]))))
    else:
        c["hi"] = _log_int(rng, 64, 16384 if kind == "append_q8" else 65536)
        c["lo"] = _log_int(rng, 1, c["hi"])
        most = 3 * (1 << 28) // (c["hi"] * kv * c["dim"])
        c["batch"] = _log_int(rng, 1, max(1, min(128, most)))
        if kind == "append_q8":
            c["chunk_hi"] = rng.choice([1, _log_int(rng, 2, 2048)])
            c["chunk_lo"] = _log_int(rng, 1, c["chunk_hi"])
    if kind == "append_q8":
        c["window"], c["sinks"] = 0, 0
    elif kind == "decode_q8" and rng.random() < 0.6:
        c["window"], c["sinks"] = 0, 0
    else:
        c["window"] = _log_int(rng, 100, 4096)
        c["sinks"] = rng.choice([0, 1, 4, 4, 16, 64])
    return c


# ---------------------------------------------------------------- lengths
def _lengths(case):
    """(context lengths, new tokens) of the case's sequences: spread over the
    logarithm, a few of them the longest; a chunk is never longer than its
    sequence."""
    g = np.random.default_rng(7000 + case["mix"])
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    ctx = np.clip(np.rint(np.exp(g.uniform(math.log(lo), math.log(hi + 0.49), b))), lo, hi)
    ctx[: b // 32] = hi
    lo, hi = case.get("chunk_lo", 1), case.get("chunk_hi", 1)
    new = np.clip(np.rint(np.exp(g.uniform(math.log(lo), math.log(hi + 0.49), b))), lo, hi)
    ctx = ctx.astype(np.int64)
    return ctx, np.minimum(new.astype(np.int64), ctx)


def _visible(case, ctx):
    """Tokens of each sequence that its last query sees."""
    if not case["window"]:
        return ctx
    first = np.minimum(case["sinks"], np.maximum(ctx - case["window"], 0))
    return np.minimum(ctx, case["window"]) + first


def work(case):
    ctx, new = _lengths(case)
    hq, hkv, d = case["heads"], case["kv_heads"], case["dim"]
    if case["kind"] == "append_q8":
        t = int(new.sum())
        blocks = int(((ctx - 1) // BLOCK - (ctx - new) // BLOCK + 1).sum())
        # new rows read, their codes written; the touched blocks' codes read and
        # written as 16-bit values; scales and table entries
        return {"bytes": 2 * t * hkv * d * (2 + 1) + 2 * blocks * hkv * BLOCK * d * (1 + 2)
                + 4 * blocks * hkv * 4 + 12 * blocks + 8 * len(ctx),
                "flops": 4.0 * t * hkv * d}
    if case["kind"] == "prefill_window":
        t = int(new.sum())
        w, s = case["window"], case["sinks"]
        pairs, union = 0, 0
        for c, n in zip(ctx.tolist(), new.tolist()):
            pos = np.arange(c - n, c)
            low = np.maximum(pos - w + 1, 0)
            pairs += int((pos - low + 1 + np.minimum(s, low)).sum())
            low0 = max(c - n - w + 1, 0)
            union += c - low0 + min(s, low0)
        return {"bytes": 2 * 2 * t * hq * d + 2 * 2 * union * hkv * d, "flops": 4.0 * pairs * hq * d}
    seen = int(_visible(case, ctx).sum())
    size = 1 if case["kind"] == "decode_q8" else 2
    extra = 8 * hkv * (seen // BLOCK) if size == 1 else 0     # a K and a V scale per block
    return {"bytes": 2 * seen * hkv * d * size + extra + 2 * 2 * len(ctx) * hq * d
            + 4 * (seen // BLOCK + len(ctx)), "flops": 4.0 * seen * hq * d}


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
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    host = np.random.default_rng([seed, case["mix"]])
    b = len(ctx)
    kind, w, s = case["kind"], case["window"], case["sinks"]

    # placement: a shuffled pool; blocks no query sees have been freed (-1)
    nblk = (ctx + BLOCK - 1) // BLOCK
    mb = int(nblk.max())
    col = np.arange(mb)[None, :]
    held = col < nblk[:, None]
    if w:
        low = np.maximum((ctx - new) - w + 1, 0)[:, None]
        held &= (col * BLOCK < s) | ((col + 1) * BLOCK > low)
    count = int(held.sum())
    nb = count + max(2, count // 10)
    tables = np.full((b, mb), -1, dtype=np.int32)
    tables[held] = host.permutation(nb)[:count].astype(np.int32)

    # keys with channels of uneven size, values with tokens of uneven size
    def fill(rows, flat):
        x = torch.randn((rows, hkv, BLOCK, d), generator=g, device=dev)
        size = torch.exp(0.5 * torch.randn((1, hkv, 1, d) if flat else (rows, hkv, BLOCK, 1),
                                           generator=g, device=dev))
        return x.mul_(size)

    st = dict(case=case, scale=1.0 / math.sqrt(d), max_ctx=int(ctx.max()), max_new=int(new.max()))
    st["block_tables"] = torch.from_numpy(tables).to(dev)
    st["context_lens"] = torch.from_numpy(ctx.astype(np.int32)).to(dev)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    st["query_start"] = torch.from_numpy(starts).to(dev)
    total = int(starts[-1])
    for name, flat in (("k", True), ("v", False)):
        x = fill(nb, flat)
        if kind in ("decode_q8", "append_q8"):
            e = _block_exponent(x.abs().amax(dim=(2, 3)))
            scale = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
            st[name + "_cache"] = _quantise(x, scale[:, :, None, None])
            st[name + "_scale"] = scale.contiguous()
        else:
            st[name + "_cache"] = x.to(dt)
        del x
    if kind == "append_q8":
        # the new tokens' own blocks; a few of the tokens are larger than what
        # their block holds, so its scale grows
        for name in ("k", "v"):
            x = torch.randn((total, hkv, d), generator=g, device=dev)
            size = torch.exp(0.8 * torch.randn((total, hkv, 1), generator=g, device=dev))
            st[name + "_new"] = (x * size).to(dt)
        first = (ctx - new) // BLOCK
        touched = (col >= first[:, None]) & (col < nblk[:, None])
        blocks = tables[touched].astype(np.int64)
        pairs = np.stack([blocks, np.arange(len(blocks))], 1)
        st["touched"] = torch.from_numpy(np.ascontiguousarray(pairs)).to(dev)
        shape = (len(blocks), hkv, BLOCK, d)
        st["k_out"] = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        st["v_out"] = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    else:
        st["q"] = torch.randn((total, hq, d), generator=g, device=dev).to(dt)
        st["out"] = torch.empty_like(st["q"])

    # what a serving loop keeps over the layers of a step: the workspace, the
    # step's plan and the calls bound to their buffers
    if own:
        import pagedattention_decode_attention_gb300 as pa
        bt, cl, qs = st["block_tables"], st["context_lens"], st["query_start"]
        if kind == "append_q8":
            st["append"] = pa.prepare_kv_append_q8(
                st["k_new"], st["v_new"], st["k_cache"], st["v_cache"], st["k_scale"],
                st["v_scale"], bt, cl, qs)
            st["read"] = pa.prepare_block_dequantize(
                st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["touched"],
                st["k_out"], st["v_out"])
        elif kind == "prefill_window":
            ws = pa.alloc_prefill_workspace(b, total, hq, hkv, d, dev)
            pa.paged_attention_prefill_window_plan(cl, qs, total, w, s, hq, hkv, d, mb,
                                                   st["scale"], dt, ws)
            st["workspace"] = ws
        else:
            ws = pa.alloc_window_workspace(b, hq, hkv, d, mb, dev)
            pa.paged_attention_decode_window_plan(cl, w, s, hq, hkv, d, mb, ws)
            if kind == "decode_q8":
                st["op"] = pa.prepare_decode_q8_run(
                    st["q"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], bt, cl,
                    w, s, st["scale"], ws, st["out"])
            else:
                st["op"] = pa.prepare_decode_window_run(
                    st["q"], st["k_cache"], st["v_cache"], bt, cl, w, s, st["scale"], ws,
                    st["out"])
    return st


# ------------------------------------------------------------ plain forms
def _gather(cache, scale, phys, off):
    """Rows [B, n, Hkv, D] in 32 bits of the tokens at (phys, off)."""
    if scale is None:
        return cache[phys, :, off].float()
    rows = cache.view(torch.uint8)[phys, :, off].view(torch.float8_e4m3fn).float()
    return rows * scale[phys][..., None]


def _plain_decode(st):
    case = st["case"]
    q, ctx, tables = st["q"], st["context_lens"].long(), st["block_tables"].long()
    b, hq, d = q.shape
    hkv = case["kv_heads"]
    w, s = case["window"], case["sinks"]
    dev = q.device
    if w:
        # the first tokens, then the window's, each token once
        last = ctx[:, None] - min(w, st["max_ctx"]) + torch.arange(min(w, st["max_ctx"]), device=dev)
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
    scores = torch.einsum("bhgd,bnhd->bhgn", q.float().view(b, hkv, hq // hkv, d), k) * st["scale"]
    del k
    scores = scores.masked_fill(~ok[:, None, None], float("-inf"))
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    v = _gather(st["v_cache"], st.get("v_scale"), phys, off)
    return torch.einsum("bhgn,bnhd->bhgd", p, v).reshape(b, hq, d).to(q.dtype)


def _plain_prefill(st):
    case = st["case"]
    q, ctx, tables = st["q"], st["context_lens"].long(), st["block_tables"].long()
    total, hq, d = q.shape
    hkv, w, s = case["kv_heads"], case["window"], case["sinks"]
    dev, b = q.device, ctx.numel()
    starts = st["query_start"].long()
    new = starts[1:] - starts[:-1]
    # rows padded to [B, longest chunk]
    slot = torch.arange(st["max_new"], device=dev)
    live = slot[None] < new[:, None]
    row = torch.where(live, starts[:-1, None] + slot[None], 0)
    qp = q.float()[row].view(b, st["max_new"], hkv, hq // hkv, d)
    pos = (ctx - new)[:, None] + slot[None]
    at = torch.arange(st["max_ctx"], device=dev)
    see = (at[None, None] <= pos[..., None]) & ((at[None, None] > pos[..., None] - w) | (at < s))
    see &= (at < ctx[:, None])[:, None]
    phys = tables[:, at // BLOCK].clamp(min=0)      # freed blocks: nothing sees them
    off = (at % BLOCK).expand(b, -1)
    k = _gather(st["k_cache"], None, phys, off)
    scores = torch.einsum("bthgd,bnhd->bhgtn", qp, k) * st["scale"]
    scores.masked_fill_(~see[:, None, None], float("-inf"))
    scores -= scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = scores.exp_()
    p /= p.sum(-1, keepdim=True)
    v = _gather(st["v_cache"], None, phys, off)
    out = torch.einsum("bhgtn,bnhd->bthgd", p, v).reshape(b, st["max_new"], hq, d)
    return out[live].to(q.dtype)


def _plain_append(st):
    ctx, tables, starts = (st[n].long() for n in ("context_lens", "block_tables", "query_start"))
    total = st["k_new"].shape[0]
    dev = ctx.device
    rows = torch.arange(total, device=dev)
    seq = torch.searchsorted(starts, rows, right=True) - 1
    new = starts[1:] - starts[:-1]
    pos = (ctx - new)[seq] + rows - starts[seq]
    phys, off = tables[seq, pos // BLOCK], pos % BLOCK
    blocks = st["touched"][:, 0]                  # every block written to, once
    nblocks = blocks.numel()
    place = torch.full((st["k_cache"].shape[0],), -1, dtype=torch.long, device=dev)
    place[blocks] = torch.arange(nblocks, device=dev)
    unit = place[phys]
    # a block that begins inside the new tokens holds nothing older
    fresh = torch.zeros(nblocks, dtype=torch.bool, device=dev)
    fresh[unit[off == 0]] = True
    held = (ctx - new)[seq] % BLOCK               # older tokens in a chunk's first block
    older = torch.zeros(nblocks, dtype=torch.long, device=dev)
    older[unit[rows == starts[seq]]] = held[rows == starts[seq]]
    older = torch.arange(BLOCK, device=dev)[None] < older[:, None]
    where = (blocks, unit, off, fresh, older)
    return {"k": _plain_quantise(st["k_cache"], st["k_scale"], st["k_new"], *where),
            "v": _plain_quantise(st["v_cache"], st["v_scale"], st["v_new"], *where),
            "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def _plain_quantise(cache, scale, new, blocks, unit, off, fresh, older):
    """Writes the rows of ``new`` into the touched blocks; the blocks' values."""
    x, codes = new.float(), cache.view(torch.uint8)
    peak = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    most = torch.zeros((blocks.numel(), x.shape[1]), device=x.device)
    most.scatter_reduce_(0, unit[:, None].expand_as(peak), peak, "amax")
    want = torch.ldexp(torch.ones_like(most), _block_exponent(most))
    old = scale[blocks]
    grown = torch.where(fresh[:, None], want, torch.maximum(old, want))
    held = codes[blocks]
    moved = held.view(torch.float8_e4m3fn).float() * (old / grown)[..., None, None]
    moved = moved.to(torch.float8_e4m3fn).view(torch.uint8)
    move = older[:, None, :, None] & (grown > old)[..., None, None]
    held = torch.where(move, moved, held)
    held[unit, :, off] = _quantise(x, grown[unit][..., None]).view(torch.uint8)
    codes[blocks] = held
    scale[blocks] = grown
    return (held.view(torch.float8_e4m3fn).float() * grown[..., None, None]).to(torch.bfloat16)


def run(state):
    kind = state["case"]["kind"]
    if own:
        import pagedattention_decode_attention_gb300 as pa
        if kind == "append_q8":
            state["append"]()
            state["read"]()
            return {"k": state["k_out"], "v": state["v_out"], "k_scale": state["k_scale"],
                    "v_scale": state["v_scale"]}
        if kind == "prefill_window":
            c = state["case"]
            return pa.paged_attention_prefill_window_run(
                state["q"], state["k_cache"], state["v_cache"], state["block_tables"],
                state["context_lens"], state["query_start"], c["window"], c["sinks"],
                state["scale"], state["workspace"], out=state["out"])
        state["op"]()
        return state["out"]
    if kind == "append_q8":
        return _plain_append(state)
    if kind == "prefill_window":
        return _plain_prefill(state)
    return _plain_decode(state)


# ------------------------------------------------------------------ exact
def _e4m3_nearest(x):
    """x rounded to the nearest e4m3 value (ties to even), in 64 bits."""
    size = np.abs(x)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.where(size > 0, size, 1.0)))
    e = np.where(np.ldexp(1.0, e.astype(int)) > size, e - 1, e)
    e = np.where(np.ldexp(1.0, (e + 1).astype(int)) <= size, e + 1, e)
    step = np.ldexp(1.0, (np.maximum(e, -6) - 3).astype(int))
    return np.clip(np.rint(x / step) * step, -448.0, 448.0)


def exact(case, seed):
    def append(case, st):
        ctx, new = _lengths(case)
        tables = st["block_tables"].cpu().numpy()
        starts = st["query_start"].cpu().numpy()
        got = {}
        for name in ("k", "v"):
            scale = st[name + "_scale"].cpu().numpy().astype(np.float64)
            rows = st[name + "_new"].float().cpu().numpy().astype(np.float64)
            held = st["touched"][:, 0]
            codes = st[name + "_cache"].view(torch.uint8)[held].view(torch.float8_e4m3fn).float()
            codes = codes.cpu().numpy().astype(np.float64)
            n = 0
            for b in range(len(ctx)):
                begin = int(ctx[b] - new[b])
                for blk in range(begin // BLOCK, (int(ctx[b]) - 1) // BLOCK + 1):
                    lo, hi = max(begin, blk * BLOCK), min(int(ctx[b]), (blk + 1) * BLOCK)
                    x = rows[starts[b] + lo - begin: starts[b] + hi - begin].transpose(1, 0, 2)
                    phys = int(tables[b, blk])
                    peak = np.abs(x).max(axis=(1, 2))
                    # smallest power of two whose 448-fold holds the peak
                    e = np.full(peak.shape, float(EXP_MIN))
                    some = peak > 0
                    e[some] = np.maximum(np.ceil(np.log2(peak[some] / 448.0)), EXP_MIN)
                    s = np.exp2(e)
                    if lo > blk * BLOCK:
                        s = np.maximum(s, scale[phys])
                        old = codes[n][:, : lo % BLOCK]
                        codes[n][:, : lo % BLOCK] = _e4m3_nearest(old * (scale[phys] / s)[:, None, None])
                    codes[n][:, lo % BLOCK: lo % BLOCK + hi - lo] = _e4m3_nearest(x / s[:, None, None])
                    codes[n] *= s[:, None, None]
                    scale[phys] = s
                    n += 1
            got[name], got[name + "_scale"] = codes, scale
        return {n: got[n] for n in ("k", "v", "k_scale", "v_scale")}

    st = prepare(case, seed)
    if case["kind"] == "append_q8":
        return append(case, st)
    ctx, new = _lengths(case)
    dev, hkv = st["q"].device, case["kv_heads"]
    w, s = case["window"], case["sinks"]
    out, row = [], 0
    for b in range(len(ctx)):
        n, t = int(ctx[b]), int(new[b])
        pos = np.arange(n - t, n)
        spans = [(0, n)]
        if w:
            low = max(n - t - w + 1, 0)
            spans = [(0, min(s, low)), (low, n)]
        at = np.concatenate([np.arange(*x) for x in spans])
        table = st["block_tables"][b].cpu().numpy().astype(np.int64)
        phys = torch.from_numpy(table[at // BLOCK]).to(dev)
        off = torch.from_numpy(at % BLOCK).to(dev)
        kv = []
        for name in ("k", "v"):
            c = st[name + "_cache"]
            if c.dtype == torch.float8_e4m3fn:
                x = c.view(torch.uint8)[phys, :, off].view(torch.float8_e4m3fn).float().double()
                x = x * st[name + "_scale"].double()[phys].unsqueeze(-1)
            else:
                x = c[phys, :, off].double()
            kv.append(x.transpose(0, 1))                         # [Hkv, n, D]
        q = st["q"][row: row + t].double()
        hide = at[None, :] > pos[:, None]
        if w:
            hide |= (at[None, :] <= pos[:, None] - w) & (at[None, :] >= s)
        hide = torch.from_numpy(hide).to(dev)
        group = q.shape[1] // hkv
        res = torch.empty_like(q)
        for h in range(hkv):
            mine = q[:, h * group: (h + 1) * group].transpose(0, 1)   # [G, T, D]
            x = mine @ kv[0][h].T * st["scale"]
            x = torch.softmax(x.masked_fill(hide, float("-inf")), -1)
            res[:, h * group: (h + 1) * group] = (x @ kv[1][h]).transpose(0, 1)
        out.append(res)
        row += t
    return torch.cat(out)
