"""Measured cases of what a prompt, or a chunk of one, needs between the projections and the output projection.

Four operators, each in a plain form (elementary torch operations in 32 bits, 64 for angles, rounded once at the end) and,
with ``own`` set, through the package's public calls:

  table   cosines and sines of a step's rows from their positions and the pairs' frequencies
  rope    rotation of queries and keys by them
  append  keys rotated on their way into a paged e4m3 cache with one power-of-two scale per (block of tokens, head), values
          beside them, and the queries of the same rows
  chunk   attention of any number of new rows per request over that cache (prompts, chunks of prompts)

A case is a dict of plain numbers; lengths and row counts of ragged batches follow from the case alone (a golden-ratio
sequence), so ``work`` counts exactly what a pass needs; values, page orders and positions come from the seed.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # One decode step of 64 requests somewhere in a long context: latency alone counts.
        dict(name="table_decode_64", op="table", n=64, rot=128, scaling="plain", reach=131072),
        # A step of prompts, positions stretched for a context 8 times the original.
        dict(name="table_prompts_16k", op="table", n=16384, rot=128, scaling="ramp", reach=262144),
        # Queries and keys of 64 decoded tokens, side by side in a fused projection of f32 GEMVs.
        dict(name="rope_decode_f32_64", op="rope", n=64, heads=40, more=8, dim=128, rot=128, start=0, pairs="half", type="f32"),
        # Queries of a step of prompts.
        dict(name="rope_prompts_bf16_16k", op="rope", n=16384, heads=64, more=16, dim=128, rot=128, start=0, pairs="half",
             type="bf16"),
        # Neighbouring pairs, rotated in the last third of each head alone, an odd number of rows.
        dict(name="rope_part_f32_1001", op="rope", n=1001, heads=24, more=0, dim=192, rot=64, start=128, pairs="neighbours",
             type="f32"),
        # The decode step's keys and values into blocks that are partly filled, and its queries, in one call.
        dict(name="append_decode_f32_64", op="append", n=64, ctx=1024, new=1, heads=32, kv=8, dim=128, block=64, rot=128,
             start=0, pairs="half", type="f32"),
        # Sixteen ragged prompts.
        dict(name="append_prompts_bf16_16", op="append", n=16, ctx=100, new=2048, heads=32, kv=8, dim=128, block=64, rot=128,
             start=0, pairs="half", type="bf16"),
        # The last rows of a prompt over a long context: few rows, so the split over its tokens is the parallelism.
        dict(name="chunk_tail_16_of_64k_bf16", op="chunk", n=1, ctx=65536, new=16, heads=32, kv=8, dim=128, block=64,
             ragged=False, type="bf16"),
        # Small pages, a head size and group that are no powers of two, rows from one to some hundred, requests of all lengths.
        dict(name="chunk_odd_9x2k_bf16", op="chunk", n=9, ctx=2001, new=301, heads=15, kv=3, dim=80, block=16, ragged=True,
             type="bf16"),
        # Prompts, some behind a cached prefix, f32 activations as the GEMVs leave them.
        dict(name="chunk_prompts_8x1k_f32", op="chunk", n=8, ctx=1024, new=1024, heads=32, kv=8, dim=128, block=64, ragged=True,
             type="f32"),
        # A chunk of 512 tokens in a serving step.
        dict(name="chunk_512_of_8k_bf16", op="chunk", n=1, ctx=8192, new=512, heads=64, kv=8, dim=128, block=64, ragged=False,
             type="bf16"),
        # A chunk of a long document: the matrix rate alone counts.
        dict(name="chunk_4k_of_16k_bf16", op="chunk", n=1, ctx=16384, new=4096, heads=64, kv=8, dim=128, block=64, ragged=False,
             type="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["table", "rope", "append", "chunk", "chunk", "chunk"])
    kind = rng.choice(["f32", "bf16"])
    dim = rng.choice([64, 80, 96, 128, 192, 256])
    rot = rng.choice([dim, dim, dim // 2, dim // 4])
    turn = dict(rot=rot, start=rng.choice([0, 0, dim - rot]), pairs=rng.choice(["half", "neighbours"]), type=kind)
    if op == "table":
        return dict(op=op, n=_log_int(rng, 1, 16384), rot=rot, scaling=rng.choice(["plain", "linear", "ramp"]),
                    reach=_log_int(rng, 4096, 1048576))
    kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    block = rng.choice([16, 32, 64, 128])
    if op == "rope":
        return dict(op=op, n=_log_int(rng, 1, 8192), heads=kv * group, more=rng.choice([0, kv, 2 * kv]), dim=dim, **turn)
    if op == "append":
        n = _log_int(rng, 1, 64)
        return dict(op=op, n=n, ctx=rng.randint(0, 700), new=_log_int(rng, 1, max(1, 8192 // n)), heads=kv * group, kv=kv, dim=dim,
                    block=block, **turn)
    n = _log_int(rng, 1, 16)
    new = _log_int(rng, 1, max(1, 4096 // n))
    ctx = new + _log_int(rng, 1, max(64, min(65536, 2 ** 35 // (n * new * kv * group * max(dim, 128)))))
    if rng.random() < 0.3:
        ctx = new  # prompts without a context
    return dict(op=op, n=n, ctx=ctx, new=new, heads=kv * group, kv=kv, dim=dim, block=block, ragged=rng.random() < 0.6, type=kind)


# ---------------------------------------------------------------- what a case's sizes are
def _spread(i, most):
    """Lengths of a ragged batch: the longest first, the rest evenly spread over 0..most."""
    return most if i == 0 else int(most * ((i * 0.6180339887498949) % 1.0))


def _sizes(c):
    """(cached tokens before the call, new tokens) of each request."""
    n = c["n"]
    if c["op"] == "append":
        return [_spread(n - 1 - i, c["ctx"]) for i in range(n)], [max(1, _spread(i, c["new"])) for i in range(n)]
    new = [max(1, _spread(i, c["new"])) if c["ragged"] else c["new"] for i in range(n)]
    total = [_spread(n - i if i else 0, c["ctx"]) if c["ragged"] else c["ctx"] for i in range(n)]
    return [max(0, t - r) for t, r in zip(total, new)], new


def _ceil(a, b):
    return -(-a // b)


def work(c):
    if c["op"] == "table":
        return {"bytes": c["n"] * (4 + 4 * c["rot"]) + 4 * c["rot"], "flops": 10 * c["n"] * c["rot"]}
    es = 4 if c["type"] == "f32" else 2
    if c["op"] == "rope":
        return {"bytes": c["n"] * (2 * c["heads"] * c["dim"] * es + 4 * c["rot"]), "flops": 3 * c["n"] * c["heads"] * c["rot"]}
    ctx, new = _sizes(c)
    t = sum(new)
    if c["op"] == "append":
        runs = sum(_ceil(a + b, c["block"]) - a // c["block"] for a, b in zip(ctx, new))
        return {"bytes": t * (8 + 4 * c["rot"] + 2 * c["kv"] * c["dim"] * (es + 1) + 2 * c["heads"] * c["dim"] * es)
                + 2 * runs * c["kv"] * 4,
                "flops": t * (4 * c["kv"] * c["dim"] + 3 * (c["heads"] + c["kv"]) * c["rot"])}
    held = sum(a + b for a, b in zip(ctx, new))
    pages = sum(_ceil(a + b, c["block"]) for a, b in zip(ctx, new))
    pairs = sum(a * b + b * (b + 1) // 2 for a, b in zip(ctx, new))
    return {"bytes": 2 * held * c["kv"] * c["dim"] + 2 * pages * c["kv"] * 4 + 4 * pages + t * c["heads"] * (2 * c["dim"] * es + 4),
            "flops": 4 * pairs * c["heads"] * c["dim"]}


# ---------------------------------------------------------------- inputs
BASE, ORIGINAL = 500000.0, 32768  # frequencies' base, tokens of the context that a stretched one was made from
FAST, SLOW = 32.0, 1.0            # ramp: pairs with more turns than FAST over the original context stay, with fewer than SLOW are stretched


def _frequencies(rot, scaling, reach):
    """Radians a token of each pair."""
    plain = [BASE ** (-2.0 * i / rot) for i in range(rot // 2)]
    factor = max(1.0, reach / ORIGINAL)
    if scaling == "plain":
        return plain
    if scaling == "linear":
        return [f / factor for f in plain]
    at = [rot * math.log(ORIGINAL / (turns * 2.0 * math.pi)) / (2.0 * math.log(BASE)) for turns in (FAST, SLOW)]
    low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(rot // 2)]
    return [f / factor * r + f * (1.0 - r) for f, r in zip(plain, ramp)]


def _cos_sin(positions, rot):
    """A step's table as its first call leaves it: [rows, 2, rot / 2]."""
    f = torch.tensor(_frequencies(rot, "plain", 0), dtype=torch.float64, device=DEV)
    angle = positions.double()[:, None] * f
    return torch.stack([torch.cos(angle), torch.sin(angle)], 1).float().contiguous()


def _pow2_scale(amax):
    """The smallest power of two s, at least 2^-126, with amax <= 448 s."""
    f, x = torch.frexp(amax)
    e = torch.where(f <= 0.875, x - 9, x - 8).clamp(min=-126)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, torch.full_like(e, -126)))


def _cache(blocks, c, gen):
    """One pool of e4m3 codes and scales, as earlier steps left it: N(0, 1) times a magnitude of each block and head."""
    codes = torch.empty((blocks, c["kv"], c["block"], c["dim"]), dtype=torch.uint8, device=DEV)
    scales = torch.empty((blocks, c["kv"]), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 27) // (c["kv"] * c["block"] * c["dim"]))
    for b in range(0, blocks, step):
        e = min(blocks, b + step)
        x = torch.randn((e - b, c["kv"], c["block"], c["dim"]), device=DEV, generator=gen)
        x *= torch.exp2(torch.randint(-1, 2, (e - b, c["kv"], 1, 1), device=DEV, generator=gen).float())
        s = _pow2_scale(x.abs().amax((2, 3)))
        codes[b:e] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[b:e] = s
    return codes, scales


def _table(lens, block, width, blocks, gen):
    """A block table of shuffled pages for `lens` tokens a request."""
    order = torch.randperm(blocks, device=DEV, generator=gen).to(torch.int32)
    have = torch.tensor([_ceil(a, block) for a in lens], device=DEV)
    first = torch.cumsum(have, 0) - have
    at = torch.arange(width, device=DEV)
    index = (first[:, None] + at).clamp(max=blocks - 1)
    return torch.where(at < have[:, None], order[index], torch.full_like(order[index], -1)).contiguous()


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if c["op"] == "table":
        s = dict(c=c, positions=torch.randint(0, c["reach"], (c["n"],), device=DEV, generator=gen, dtype=torch.int32),
                 freqs=torch.tensor(_frequencies(c["rot"], c["scaling"], c["reach"]), dtype=torch.float64, device=DEV),
                 scale=1.0 + 0.1 * math.log(max(1.0, c["reach"] / ORIGINAL)) if c["scaling"] == "ramp" else 1.0)
        if own:
            from fp8_block_scaled_fp8blk_gb300 import ops
            freqs, _ = ops.rope_frequencies(c["rot"], BASE, c["scaling"], factor=max(1.0, c["reach"] / ORIGINAL),
                                            original_len=ORIGINAL, low=SLOW, high=FAST)
            s["turns"] = ops.rope_turns(freqs, DEV)
            s["out"] = torch.empty((c["n"], 2, c["rot"] // 2), dtype=torch.float32, device=DEV)
        return s
    kind = TYPES[c["type"]]
    if c["op"] == "rope":
        qkv = torch.randn((c["n"], c["heads"] + c["more"], c["dim"]), device=DEV, generator=gen).to(kind)
        positions = torch.randint(0, 131072, (c["n"],), device=DEV, generator=gen, dtype=torch.int32)
        s = dict(c=c, x=qkv[:, : c["heads"]], cos_sin=_cos_sin(positions, c["rot"]))
        if own:
            s["out"] = torch.empty((c["n"], c["heads"], c["dim"]), dtype=kind, device=DEV)
        return s
    ctx, new = _sizes(c)
    total = [a + b for a, b in zip(ctx, new)]
    width = max(1, max(_ceil(t, c["block"]) for t in total))
    blocks = max(1, sum(_ceil(t, c["block"]) for t in total))
    table = _table(total, c["block"], width, blocks, gen)
    k_codes, k_scales = _cache(blocks, c, gen)
    v_codes, v_scales = _cache(blocks, c, gen)
    s = dict(c=c, table=table, k_codes=k_codes, k_scales=k_scales, v_codes=v_codes, v_scales=v_scales)
    if c["op"] == "append":
        t = sum(new)
        qkv = torch.randn((t, c["heads"] + 2 * c["kv"], c["dim"]), device=DEV, generator=gen).to(kind)
        s["q"] = qkv[:, : c["heads"]]
        s["k"], s["v"] = qkv[:, c["heads"]: c["heads"] + c["kv"]], qkv[:, c["heads"] + c["kv"]:]
        pos = torch.cat([torch.arange(a, a + b) for a, b in zip(ctx, new)]).to(DEV)
        req = torch.repeat_interleave(torch.arange(c["n"]), torch.tensor(new)).to(DEV)
        s["slots"] = table[req, pos // c["block"]].long() * c["block"] + pos % c["block"]
        s["cos_sin"] = _cos_sin(pos, c["rot"])
        s["runs"] = sum(_ceil(a + b, c["block"]) - a // c["block"] for a, b in zip(ctx, new))
        if own:
            s["q_out"] = torch.empty((t, c["heads"], c["dim"]), dtype=kind, device=DEV)
        return s
    s["q"] = (1.5 * torch.randn((sum(new), c["heads"], c["dim"]), device=DEV, generator=gen)).to(kind)
    s["lens"] = torch.tensor(total, dtype=torch.int32, device=DEV)
    starts = [0]
    for r in new:
        starts.append(starts[-1] + r)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    s["most"] = max(new)
    s["scale"] = 1.0 / math.sqrt(c["dim"])
    if own:
        from fp8_block_scaled_fp8blk_gb300 import ops
        s["ws"] = ops.kv_attn_chunk_workspace(c["heads"], c["kv"], c["dim"], DEV)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["c"]["op"]
    if own:
        return {"table": _table_own, "rope": _rope_own, "append": _append_own, "chunk": _chunk_own}[op](s)
    return {"table": _table_plain, "rope": _rope_plain, "append": _append_plain, "chunk": _chunk_plain}[op](s)


def _table_own(s):
    from fp8_block_scaled_fp8blk_gb300 import ops
    return ops.fp8blk_rope_table(s["positions"], s["turns"], s["scale"], out=s["out"])


def _table_plain(s):
    angle = s["positions"].double()[:, None] * s["freqs"]  # far positions need the 64 bits
    return (torch.stack([torch.cos(angle), torch.sin(angle)], 1) * s["scale"]).float()


def _rope_own(s):
    from fp8_block_scaled_fp8blk_gb300 import ops
    return ops.fp8blk_rope(s["x"], s["cos_sin"], interleaved=s["c"]["pairs"] == "neighbours", start=s["c"]["start"], out=s["out"])


def _rotated(x, cos_sin, c):
    """x [rows, heads, dim] in 32 bits with its rotated part turned."""
    x, a, half = x.float(), c["start"], c["rot"] // 2
    cos, sin = cos_sin[:, None, 0], cos_sin[:, None, 1]
    part = x[:, :, a: a + c["rot"]]
    if c["pairs"] == "half":
        u, v = part[:, :, :half], part[:, :, half:]
        part = torch.cat([u * cos - v * sin, v * cos + u * sin], 2)
    else:
        u, v = part[:, :, 0::2], part[:, :, 1::2]
        part = torch.stack([u * cos - v * sin, v * cos + u * sin], 3).flatten(2)
    return torch.cat([x[:, :, :a], part, x[:, :, a + c["rot"]:]], 2)


def _rope_plain(s):
    return _rotated(s["x"], s["cos_sin"], s["c"]).to(s["x"].dtype)


def _append_own(s):
    from fp8_block_scaled_fp8blk_gb300 import ops
    ops.fp8blk_kv_append_rope(s["k"], s["v"], s["slots"], s["cos_sin"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"],
                              interleaved=s["c"]["pairs"] == "neighbours", start=s["c"]["start"], q=s["q"], q_out=s["q_out"])
    return dict(_pools(s), q=s["q_out"])


def _pools(s):
    return dict(k=s["k_codes"].view(torch.float8_e4m3fn), ks=s["k_scales"], v=s["v_codes"].view(torch.float8_e4m3fn), vs=s["v_scales"])


def _append_plain(s):
    c, block, slots = s["c"], s["c"]["block"], s["slots"]
    page, off = slots // block, slots % block
    head = torch.ones_like(slots, dtype=torch.bool)
    head[1:] = page[1:] != page[:-1]
    lead = torch.argsort(~head, stable=True)[: s["runs"]]  # first token of each run of tokens in one block
    run_of = torch.cumsum(head, 0) - 1

    def write(x, codes, scales):
        peak = torch.zeros((s["runs"], x.shape[1]), device=x.device)
        peak.scatter_reduce_(0, run_of[:, None].expand(x.shape[:2]), x.abs().amax(2), "amax")
        need = _pow2_scale(peak)
        old = scales[page[lead]]
        scale = torch.where((off[lead] > 0)[:, None], torch.maximum(old, need), need)
        held = codes[page[lead]]  # rows that were there follow the larger scale
        moved = (held.view(torch.float8_e4m3fn).float() * (old / scale)[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        there = torch.arange(block, device=x.device) < off[lead][:, None]
        codes[page[lead]] = torch.where(there[:, None, :, None] & (old != scale)[:, :, None, None], moved, held)
        scales[page[lead]] = scale
        codes[page, :, off] = (x / scale[run_of][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)

    write(_rotated(s["k"], s["cos_sin"], c), s["k_codes"], s["k_scales"])
    write(s["v"].float(), s["v_codes"], s["v_scales"])
    return dict(_pools(s), q=_rotated(s["q"], s["cos_sin"], c).to(s["q"].dtype))


def _chunk_own(s):
    from fp8_block_scaled_fp8blk_gb300 import ops
    ops.fp8blk_kv_attn_chunk(s["q"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["table"], s["lens"], s["starts"],
                             s["scale"], s["ws"], out=s["out"], lse=s["lse"])
    return dict(out=s["out"], lse=s["lse"])


def _chunk_plain(s):
    c, q, m = s["c"], s["q"], s["most"]
    n, kv, dim = c["n"], c["kv"], c["dim"]
    group, width = c["heads"] // kv, s["table"].shape[1]
    page = s["table"].long().clamp(min=0)

    def tokens(codes, scales):  # [n, kv, width * block, dim]
        x = codes[page].view(torch.float8_e4m3fn).float() * scales[page][:, :, :, None, None]
        return x.transpose(1, 2).reshape(n, kv, width * c["block"], dim)

    rows = (s["starts"][1:] - s["starts"][:-1]).long()
    at = torch.arange(m, device=q.device)
    index = (s["starts"][:-1].long()[:, None] + at).clamp(max=q.shape[0] - 1)
    x = q[index].float().view(n, m, kv, group, dim).permute(0, 2, 1, 3, 4).reshape(n, kv, m * group, dim)
    score = torch.matmul(x, tokens(s["k_codes"], s["k_scales"]).transpose(2, 3))
    score *= s["scale"]
    last = s["lens"].long()[:, None] - rows[:, None] + at  # the position of each row: it sees what is at or before it
    hidden = torch.arange(width * c["block"], device=q.device) > last[:, :, None]
    score.view(n, kv, m, group, -1).masked_fill_(hidden[:, None, :, None], float("-inf"))
    top = score.amax(3, keepdim=True)
    score -= top
    weight = score.exp_()
    total = weight.sum(3, keepdim=True)
    past = torch.arange(width * c["block"], device=q.device) >= s["lens"].long()[:, None]
    value = torch.where(past[:, None, :, None], 0.0, tokens(s["v_codes"], s["v_scales"]))
    out = torch.matmul(weight, value) / total
    lse = torch.log(total) + top
    out = out.view(n, kv, m, group, dim).permute(0, 2, 1, 3, 4).reshape(n, m, c["heads"], dim)
    lse = lse.view(n, kv, m, group).permute(0, 2, 1, 3).reshape(n, m, c["heads"])
    req = torch.searchsorted(s["starts"][1:].contiguous(), torch.arange(q.shape[0], device=q.device, dtype=torch.int32), right=True)
    row = torch.arange(q.shape[0], device=q.device) - s["starts"].long()[req]
    return dict(out=out[req, row].to(q.dtype), lse=lse[req, row])


# ---------------------------------------------------------------- the definitions in 64 bits
def _e4m3_values():
    """The 256 codes' values from their bit fields."""
    out = []
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        v = math.nan if (e, f) == (15, 7) else math.ldexp(f, -9) if e == 0 else math.ldexp(8 + f, e - 10)
        out.append(-v if b & 128 else v)
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def _nearest_e4m3(x):
    """x in 64 bits to the nearest e4m3 value, halves to the even code, beyond the range to its end."""
    grid = _e4m3_values()[:127]
    a = x.abs().clamp(max=448.0)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, 126)
    lo = hi - 1
    down, up = a - grid[lo], grid[hi] - a
    code = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return torch.copysign(grid[code], x)


def _turned(x, cos_sin, c):
    """The rotation pair by pair, as complex numbers."""
    z = torch.complex(cos_sin[:, 0].double(), cos_sin[:, 1].double())[:, None]
    y, i = x.double().clone(), torch.arange(c["rot"] // 2, device=x.device)
    first, second = (i, i + c["rot"] // 2) if c["pairs"] == "half" else (2 * i, 2 * i + 1)
    p = torch.complex(y[:, :, c["start"] + first], y[:, :, c["start"] + second]) * z
    y[:, :, c["start"] + first], y[:, :, c["start"] + second] = p.real, p.imag
    return y


def exact(c, seed):
    global own
    was, own = own, False
    s = prepare(c, seed)
    own = was
    if c["op"] == "table":
        z = torch.polar(torch.full((), s["scale"], dtype=torch.float64, device=DEV), torch.outer(s["positions"].double(), s["freqs"]))
        return torch.stack([z.real, z.imag], 1)
    if c["op"] == "rope":
        return _turned(s["x"], s["cos_sin"], c)
    ctx, new = _sizes(c)
    block, value = c["block"], _e4m3_values()
    if c["op"] == "append":
        out = dict(k=None, ks=None, v=None, vs=None, q=_turned(s["q"], s["cos_sin"], c))
        for x, codes, scales, name in ((_turned(s["k"], s["cos_sin"], c), s["k_codes"], s["k_scales"], "k"),
                                       (s["v"].double(), s["v_codes"], s["v_scales"], "v")):
            held, scale, at = value[codes.long()], scales.double(), 0
            for i in range(c["n"]):
                p = ctx[i]
                while p < ctx[i] + new[i]:
                    page, off = int(s["table"][i, p // block]), p % block
                    take = min(block - off, ctx[i] + new[i] - p)
                    rows = x[at: at + take].transpose(0, 1)
                    e = torch.ceil(torch.log2(rows.abs().amax((1, 2)) / 448.0)).clamp(min=-126)
                    old, want = scale[page].clone(), torch.exp2(e)
                    want = torch.maximum(old, want) if off else want
                    if off:
                        held[page, :, :off] = _nearest_e4m3(held[page, :, :off] * (old / want)[:, None, None])
                    held[page, :, off: off + take] = _nearest_e4m3(rows / want[:, None, None])
                    scale[page] = want
                    at, p = at + take, p + take
            out[name], out[name + "s"] = held, scale
        return out
    outs, lses, starts = [], [], s["starts"].tolist()
    group = c["heads"] // c["kv"]
    for i in range(c["n"]):
        length, rows = ctx[i] + new[i], new[i]
        page = s["table"][i, : _ceil(length, block)].long()

        def tokens(codes, scales):
            x = value[codes[page].long()] * scales[page].double()[:, :, None, None]
            return x.permute(1, 0, 2, 3).reshape(c["kv"], -1, c["dim"])[:, :length]

        k, v = tokens(s["k_codes"], s["k_scales"]), tokens(s["v_codes"], s["v_scales"])
        for r in range(0, rows, 64):
            e = min(rows, r + 64)
            seen = length - rows + e
            q = s["q"][starts[i] + r: starts[i] + e].double().view(e - r, c["kv"], group, c["dim"])
            score = torch.einsum("rhgd,htd->rhgt", q, k[:, :seen]) * s["scale"]
            last = length - rows + torch.arange(r, e, device=DEV)
            score = torch.where(torch.arange(seen, device=DEV) <= last[:, None, None, None], score, -math.inf)
            lse = torch.logsumexp(score, 3)
            out = torch.einsum("rhgt,htd->rhgd", torch.exp(score - lse[..., None]), v[:, :seen])
            outs.append(out.reshape(e - r, c["heads"], c["dim"]))
            lses.append(lse.reshape(e - r, c["heads"]))
    return dict(out=torch.cat(outs), lse=torch.cat(lses))
