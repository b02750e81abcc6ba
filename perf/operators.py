"""Measured cases of the serving operators around the GEMVs of a decode or verify step.

Four operators, each in a plain form (elementary torch operations in 32 bits, rounded once at the end) and, with
``own`` set, through the package's public calls:

  map       block tables, slots and positions of a paged cache, from request lengths on the device
  append    keys and values into a paged e4m3 cache with one power-of-two scale per (block of tokens, head)
  attn      attention of 1..8 new rows per request over that cache (decode and speculative verify)
  logprobs  log probability, rank and entropy of given tokens, with the top alternatives

A case is a dict of plain numbers; lengths and row counts of ragged batches follow from the case alone (a golden-ratio
sequence), so ``work`` counts exactly what a pass needs; values, page orders and targets come from the seed.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # A decode step of 64 running requests: one new token each; latency alone counts.
        dict(name="map_decode_64", op="map", n=64, ctx=8192, new=1, block=64),
        # Admission of 512 prompts of up to 8192 tokens, some behind a cached prefix: 1.8 million slots.
        dict(name="map_prompts_512", op="map", n=512, ctx=512, new=8192, block=16),
        # The same decode step's keys and values (f32, as the GEMVs write them) into blocks already partly filled.
        dict(name="append_decode_f32_64", op="append", n=64, ctx=1024, new=1, heads=32, kv=8, dim=128, block=64,
             type="f32"),
        # Sixteen ragged prompts, bf16.
        dict(name="append_prompts_bf16_16", op="append", n=16, ctx=100, new=2048, heads=32, kv=8, dim=128, block=64,
             type="bf16"),
        # One request in a short chat, f32 activations as the GEMVs leave them: latency of a single decode step.
        dict(name="attn_decode_1x1k_f32", op="attn", n=1, ctx=1023, m=1, heads=32, kv=8, dim=128, block=64,
             ragged=False, type="f32"),
        # One request with a long context: the split over its tokens is all the parallelism there is.
        dict(name="attn_decode_1x128k_bf16", op="attn", n=1, ctx=131071, m=1, heads=64, kv=8, dim=128, block=64,
             ragged=False, type="bf16"),
        # A serving batch in decode, ragged lengths.
        dict(name="attn_decode_64x8k_bf16", op="attn", n=64, ctx=8192, m=1, heads=64, kv=8, dim=128, block=64,
             ragged=True, type="bf16"),
        # A batch in speculative verify, eight rows a request, f32.
        dict(name="attn_verify_16x16k_f32", op="attn", n=16, ctx=16384, m=8, heads=32, kv=8, dim=128, block=128,
             ragged=True, type="f32"),
        # Small pages, a head size and group that are no powers of two, 1..5 rows, requests that have nothing cached.
        dict(name="attn_odd_33x2k_bf16", op="attn", n=33, ctx=2001, m=5, heads=15, kv=3, dim=80, block=16,
             ragged=True, type="bf16"),
        # The verify window's eight rows of the 131072-entry head.
        dict(name="logprobs_verify_8_f32", op="logprobs", n=8, vocab=131072, top=5, type="f32"),
        # A short scoring call, bf16 logits (many ties), a vocabulary that is no multiple of anything.
        dict(name="logprobs_odd_77_bf16", op="logprobs", n=77, vocab=100003, top=10, type="bf16"),
        # Scoring whole documents: bandwidth alone counts.
        dict(name="logprobs_score_2048_f32", op="logprobs", n=2048, vocab=131072, top=20, type="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["map", "append", "attn", "attn", "logprobs"])
    if op == "map":
        n = _log_int(rng, 1, 512)
        return dict(op=op, n=n, ctx=rng.randint(0, 8192), new=_log_int(rng, 1, 4096), block=rng.choice([16, 32, 64, 128]))
    kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    dim = rng.choice([64, 80, 96, 128, 192, 256])
    block = rng.choice([16, 32, 64, 128])
    kind = rng.choice(["f32", "bf16"])
    if op == "append":
        n = _log_int(rng, 1, 64)
        new = _log_int(rng, 1, max(1, 8192 // n))
        return dict(op=op, n=n, ctx=rng.randint(0, 700), new=new, heads=kv * group, kv=kv, dim=dim, block=block, type=kind)
    if op == "attn":
        n = _log_int(rng, 1, 64)
        ctx = _log_int(rng, 1, max(64, min(100000, 2 ** 28 // (n * kv * dim))))
        return dict(op=op, n=n, ctx=ctx, m=rng.randint(1, 8), heads=kv * group, kv=kv, dim=dim, block=block,
                    ragged=rng.random() < 0.7, type=kind)
    return dict(op=op, n=_log_int(rng, 1, 1024), vocab=_log_int(rng, 1000, 131072), top=rng.randint(0, 20), type=kind)


# ---------------------------------------------------------------- what a case's sizes are
def _spread(i, most):
    """Lengths of a ragged batch: the longest first, the rest evenly spread over 0..most."""
    return most if i == 0 else int(most * ((i * 0.6180339887498949) % 1.0))


def _sizes(c):
    """(cached tokens before the call, new tokens) of each request."""
    n = c["n"]
    if c["op"] == "map":
        new = [max(1, _spread(i, c["new"])) for i in range(n)]
        return [_spread(n - 1 - i, c["ctx"]) for i in range(n)], new
    if c["op"] == "append":
        new = [max(1, _spread(i, c["new"])) for i in range(n)]
        return [_spread(n - 1 - i, c["ctx"]) for i in range(n)], new
    rows = [1 + (5 * i + c["m"] - 1) % c["m"] if c["ragged"] else c["m"] for i in range(n)]
    total = [_spread(i, c["ctx"]) if c["ragged"] else c["ctx"] for i in range(n)]
    return [max(0, t - r) for t, r in zip(total, rows)], [min(t, r) for t, r in zip(total, rows)]


def _rows(c):
    """Query rows of each request of an attention case: a request that holds fewer tokens leaves its first rows empty."""
    return [1 + (5 * i + c["m"] - 1) % c["m"] if c["ragged"] else c["m"] for i in range(c["n"])]


def _ceil(a, b):
    return -(-a // b)


def work(c):
    if c["op"] == "logprobs":
        es = 4 if c["type"] == "f32" else 2
        return {"bytes": c["n"] * (c["vocab"] * es + 4 + 12 + 8 * c["top"]), "flops": 6 * c["n"] * c["vocab"]}
    ctx, new = _sizes(c)
    if c["op"] == "map":
        taken = sum(_ceil(a + b, c["block"]) - _ceil(a, c["block"]) for a, b in zip(ctx, new))
        return {"bytes": 8 * c["n"] + 8 * c["n"] + 8 * taken + 12 * sum(new), "flops": 0}
    es = 4 if c["type"] == "f32" else 2
    if c["op"] == "append":
        runs = sum(_ceil(a + b, c["block"]) - a // c["block"] for a, b in zip(ctx, new))
        t = sum(new)
        return {"bytes": t * 8 + 2 * t * c["kv"] * c["dim"] * (es + 1) + 2 * runs * c["kv"] * 4,
                "flops": 4 * t * c["kv"] * c["dim"]}
    rows = _rows(c)
    held = sum(a + b for a, b in zip(ctx, new))
    pages = sum(_ceil(a + b, c["block"]) for a, b in zip(ctx, new))
    pairs = sum(sum(max(0, a + b - r + i + 1) for i in range(r)) for a, b, r in zip(ctx, new, rows))
    return {"bytes": 2 * held * c["kv"] * c["dim"] + 2 * pages * c["kv"] * 4 + 4 * pages
            + sum(rows) * c["heads"] * (2 * c["dim"] * es + 4),
            "flops": 4 * pairs * c["heads"] * c["dim"]}


# ---------------------------------------------------------------- inputs
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


def _table(ctx, block, width, blocks, gen, spare=0):
    """A block table of shuffled pages for `ctx` tokens a request, and the pages that are left over."""
    order = torch.randperm(blocks, device=DEV, generator=gen).to(torch.int32)
    have = torch.tensor([_ceil(a, block) for a in ctx], device=DEV)
    first = torch.cumsum(have, 0) - have
    at = torch.arange(width, device=DEV)
    index = (first[:, None] + at).clamp(max=blocks - 1)
    table = torch.where(at < have[:, None], order[index], torch.full_like(order[index], -1))
    return table.contiguous(), order, int(sum(_ceil(a, block) for a in ctx))


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if c["op"] == "logprobs":
        kind = TYPES[c["type"]]
        logits = torch.empty((c["n"], c["vocab"]), dtype=kind, device=DEV)
        for r in range(0, c["n"], 256):
            e = min(c["n"], r + 256)
            logits[r:e] = 2.5 * torch.randn((e - r, c["vocab"]), device=DEV, generator=gen)
        targets = torch.randint(0, c["vocab"], (c["n"],), device=DEV, generator=gen)
        up = torch.where(torch.rand(c["n"], device=DEV, generator=gen) < 0.7, 11.0, 0.0)  # most drafted tokens are likely ones
        row = torch.arange(c["n"], device=DEV)
        logits[row, targets] = (logits[row, targets].float() + up).to(kind)
        s = dict(c=c, logits=logits, targets=targets.to(torch.int32))
        if own:
            from fp8_block_scaled_fp8blk_gb300 import ops
            s["out"] = ops.token_logprobs_buffers(c["n"], c["top"], DEV)
        return s
    ctx, new = _sizes(c)
    if c["op"] == "map":
        width = max(_ceil(a + b, c["block"]) for a, b in zip(ctx, new))
        blocks = sum(_ceil(a + b, c["block"]) for a, b in zip(ctx, new)) + 32
        table, order, head = _table(ctx, c["block"], width, blocks, gen)
        most = _ceil(sum(new), 64) * 64  # a step that is captured once has room for a fixed number of tokens
        s = dict(c=c, ctx=torch.tensor(ctx, dtype=torch.int32, device=DEV), new=torch.tensor(new, dtype=torch.int32, device=DEV),
                 table=table, free=order, head=torch.tensor([head], dtype=torch.int32, device=DEV), most=most)
        if own:
            from fp8_block_scaled_fp8blk_gb300 import ops
            s["out"] = ops.kv_map_buffers(c["n"], most, DEV)
        return s
    total = [a + b for a, b in zip(ctx, new)]
    width = max(1, max(_ceil(t, c["block"]) for t in total))
    blocks = max(1, sum(_ceil(t, c["block"]) for t in total))
    table, _, _ = _table(total, c["block"], width, blocks, gen)
    k_codes, k_scales = _cache(blocks, c, gen)
    v_codes, v_scales = _cache(blocks, c, gen)
    s = dict(c=c, table=table, k_codes=k_codes, k_scales=k_scales, v_codes=v_codes, v_scales=v_scales)
    kind = TYPES[c["type"]]
    if c["op"] == "append":
        t = sum(new)
        qkv = torch.randn((t, c["heads"] + 2 * c["kv"], c["dim"]), device=DEV, generator=gen).to(kind)
        s["k"], s["v"] = qkv[:, c["heads"]: c["heads"] + c["kv"]], qkv[:, c["heads"] + c["kv"]:]
        pos = torch.cat([torch.arange(a, a + b) for a, b in zip(ctx, new)]).to(DEV)
        req = torch.repeat_interleave(torch.arange(c["n"]), torch.tensor(new)).to(DEV)
        s["slots"] = table[req, pos // c["block"]].long() * c["block"] + pos % c["block"]
        s["runs"] = sum(_ceil(a + b, c["block"]) - a // c["block"] for a, b in zip(ctx, new))
        return s
    rows = _rows(c)
    s["q"] = 1.5 * torch.randn((sum(rows), c["heads"], c["dim"]), device=DEV, generator=gen)
    s["q"] = s["q"].to(kind)
    s["lens"] = torch.tensor(total, dtype=torch.int32, device=DEV)
    starts = [0]
    for r in rows:
        starts.append(starts[-1] + r)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    s["scale"] = 1.0 / math.sqrt(c["dim"])
    if own:
        from fp8_block_scaled_fp8blk_gb300 import ops
        s["ws"] = ops.kv_attn_workspace(c["n"], c["m"], c["heads"], c["kv"], c["dim"], DEV)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["c"]["op"]
    if own:
        return {"map": _map_own, "append": _append_own, "attn": _attn_own, "logprobs": _logprobs_own}[op](s)
    return {"map": _map_plain, "append": _append_plain, "attn": _attn_plain, "logprobs": _logprobs_plain}[op](s)


def _map_own(s):
    from fp8_block_scaled_fp8blk_gb300 import ops
    r = ops.fp8blk_kv_map(s["ctx"], s["new"], s["table"], s["free"], s["head"], s["c"]["block"], s["most"], out=s["out"])
    return dict(table=s["table"], lens=r.seq_lens, starts=r.q_starts, slots=r.slots, positions=r.positions, head=r.free_head)


def _map_plain(s):
    block, most = s["c"]["block"], s["most"]
    ctx, new, table = s["ctx"].long(), s["new"].long(), s["table"]
    lens = ctx + new
    held, wanted = (ctx + block - 1) // block, (lens + block - 1) // block
    taken = wanted - held
    first = s["head"].long() + torch.cumsum(taken, 0) - taken
    at = torch.arange(table.shape[1], device=table.device)
    fresh = (at >= held[:, None]) & (at < wanted[:, None])
    page = s["free"][(first[:, None] + at - held[:, None]).clamp(0, s["free"].numel() - 1)]
    table.copy_(torch.where(fresh, page, table))
    starts = torch.cat([torch.zeros_like(lens[:1]), torch.cumsum(new, 0)])
    token = torch.arange(most, device=table.device)
    req = torch.searchsorted(starts[1:], token, right=True).clamp(max=new.numel() - 1)
    pos = ctx[req] + token - starts[req]
    live = token < starts[-1]
    index = (pos // block).clamp(0, table.shape[1] - 1)
    slots = torch.where(live, table[req, index].long() * block + pos % block, -1)
    return dict(table=table, lens=lens.int(), starts=starts.int(), slots=slots, positions=torch.where(live, pos, -1).int(),
                head=(s["head"] + taken.sum()).int())


def _append_own(s):
    from fp8_block_scaled_fp8blk_gb300 import ops
    ops.fp8blk_kv_append(s["k"], s["v"], s["slots"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
    return _pools(s)


def _pools(s):
    return dict(k=s["k_codes"].view(torch.float8_e4m3fn), ks=s["k_scales"], v=s["v_codes"].view(torch.float8_e4m3fn), vs=s["v_scales"])


def _append_plain(s):
    block, slots = s["c"]["block"], s["slots"]
    page, off = slots // block, slots % block
    head = torch.ones_like(slots, dtype=torch.bool)
    head[1:] = page[1:] != page[:-1]
    lead = torch.argsort(~head, stable=True)[: s["runs"]]  # first token of each run of tokens in one block
    run_of = torch.cumsum(head, 0) - 1
    for x, codes, scales in ((s["k"], s["k_codes"], s["k_scales"]), (s["v"], s["v_codes"], s["v_scales"])):
        x = x.float()
        good = torch.isfinite(x)
        amax = torch.where(good, x.abs(), 0.0).amax(2)
        peak = torch.zeros((s["runs"], x.shape[1]), device=x.device)
        peak.scatter_reduce_(0, run_of[:, None].expand_as(amax), amax, "amax")
        need = _pow2_scale(peak)
        old = scales[page[lead]]
        scale = torch.where((off[lead] > 0)[:, None], torch.maximum(old, need), need)
        held = codes[page[lead]]  # rows that were there follow the larger scale
        moved = (held.view(torch.float8_e4m3fn).float() * (old / scale)[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        there = torch.arange(block, device=x.device) < off[lead][:, None]
        codes[page[lead]] = torch.where(there[:, None, :, None] & (old != scale)[:, :, None, None], moved, held)
        scales[page[lead]] = scale
        y = torch.where(good, x / scale[run_of][:, :, None], float("nan"))
        codes[page, :, off] = y.to(torch.float8_e4m3fn).view(torch.uint8)
    return _pools(s)


def _attn_own(s):
    from fp8_block_scaled_fp8blk_gb300 import ops
    ops.fp8blk_kv_attn(s["q"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["table"], s["lens"], s["starts"],
                       s["c"]["m"], s["scale"], s["ws"], out=s["out"], lse=s["lse"])
    return dict(out=s["out"], lse=s["lse"])


def _attn_plain(s):
    c, q = s["c"], s["q"]
    n, m, kv, dim = c["n"], c["m"], c["kv"], c["dim"]
    group, width = c["heads"] // kv, s["table"].shape[1]
    page = s["table"].long().clamp(min=0)

    def tokens(codes, scales):  # [n, kv, width * block, dim]
        x = codes[page].view(torch.float8_e4m3fn).float() * scales[page][:, :, :, None, None]
        return x.transpose(1, 2).reshape(n, kv, width * c["block"], dim)

    rows = (s["starts"][1:] - s["starts"][:-1]).long()
    at = torch.arange(m, device=q.device)
    live = at < rows[:, None]
    index = (s["starts"][:-1].long()[:, None] + at).clamp(max=q.shape[0] - 1)
    x = q[index].float().view(n, m, kv, group, dim).permute(0, 2, 1, 3, 4).reshape(n, kv, m * group, dim)
    score = torch.matmul(x, tokens(s["k_codes"], s["k_scales"]).transpose(2, 3)) * s["scale"]
    last = s["lens"].long()[:, None] - rows[:, None] + at  # the position of each row: it sees what is at or before it
    seen = torch.arange(width * c["block"], device=q.device) <= last[:, :, None]
    seen = seen[:, None, :, None].expand(n, kv, m, group, -1).reshape(score.shape)
    score = torch.where(seen, score, float("-inf"))
    top = score.amax(3, keepdim=True)
    weight = torch.exp(score - torch.where(torch.isfinite(top), top, 0.0))
    total = weight.sum(3, keepdim=True)
    past = torch.arange(width * c["block"], device=q.device) >= s["lens"].long()[:, None]
    value = torch.where(past[:, None, :, None], 0.0, tokens(s["v_codes"], s["v_scales"]))
    out = torch.matmul(weight, value) / torch.where(total > 0, total, 1.0)
    lse = torch.log(total) + torch.where(torch.isfinite(top), top, 0.0)
    out = out.view(n, kv, m, group, dim).permute(0, 2, 1, 3, 4).reshape(n, m, c["heads"], dim)
    lse = lse.view(n, kv, m, group).permute(0, 2, 1, 3).reshape(n, m, c["heads"])
    req = torch.searchsorted(s["starts"][1:].contiguous(), torch.arange(q.shape[0], device=q.device, dtype=torch.int32), right=True)
    row = torch.arange(q.shape[0], device=q.device) - s["starts"].long()[req]
    return dict(out=out[req, row].to(q.dtype), lse=lse[req, row])


def _logprobs_own(s):
    from fp8_block_scaled_fp8blk_gb300 import ops
    r = ops.fp8blk_token_logprobs(s["logits"], s["targets"], s["c"]["top"], out=s["out"])
    return dict(logprob=r.logprob, rank=r.rank, entropy=r.entropy, ids=r.top_ids, top=r.top_logprobs)


def _logprobs_plain(s):
    x, t, k = s["logits"].float(), s["targets"].long(), s["c"]["top"]
    vocab = x.shape[1]
    peak = x.amax(1, keepdim=True)
    d = x - peak
    e = torch.exp(d)
    total = e.sum(1)
    entropy = torch.log(total) - torch.where(e > 0, e * d, 0.0).sum(1) / total
    lse = torch.log(total)[:, None]
    mine = x.gather(1, t[:, None])
    index = torch.arange(vocab, device=x.device)
    rank = ((x > mine) | ((x == mine) & (index < t[:, None]))).sum(1)
    bits = (x + 0.0).view(torch.int32)
    key = (torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF).long() << 32) | (vocab - 1 - index)
    ids = vocab - 1 - (torch.topk(key, k, 1).values & 0xFFFFFFFF)
    return dict(logprob=(mine - peak - lse)[:, 0], rank=rank.int(), entropy=entropy, ids=ids.int(), top=x.gather(1, ids) - peak - lse)


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
    return torch.where(torch.isnan(x), x, torch.copysign(grid[code], x))


def exact(c, seed):
    if c["op"] == "map":
        return None  # whole numbers
    global own
    was, own = own, False
    s = prepare(c, seed)
    own = was
    if c["op"] == "logprobs":
        logprob, entropy, top = [], [], []
        for r in range(0, c["n"], 128):
            x = s["logits"][r: r + 128].double()
            lse = torch.logsumexp(x, 1, keepdim=True)
            logp = x - lse
            logprob.append(logp.gather(1, s["targets"][r: r + 128].long()[:, None])[:, 0])
            entropy.append(-(logp.exp() * logp).sum(1))
            top.append(logp.topk(c["top"], 1).values)
        return dict(logprob=torch.cat(logprob), rank=None, entropy=torch.cat(entropy), ids=None, top=torch.cat(top))
    ctx, new = _sizes(c)
    block, value = c["block"], _e4m3_values()
    if c["op"] == "append":
        out, at = {}, 0
        for x, codes, scales, name in ((s["k"], s["k_codes"], s["k_scales"], "k"), (s["v"], s["v_codes"], s["v_scales"], "v")):
            held, scale, at = value[codes.long()], scales.double(), 0
            for i in range(c["n"]):
                p = ctx[i]
                while p < ctx[i] + new[i]:
                    page, off = int(s["table"][i, p // block]), p % block
                    take = min(block - off, ctx[i] + new[i] - p)
                    rows = x[at: at + take].double().transpose(0, 1)
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
        length, rows = ctx[i] + new[i], starts[i + 1] - starts[i]
        page = s["table"][i, : _ceil(length, block)].long()

        def tokens(codes, scales):
            x = value[codes[page].long()] * scales[page].double()[:, :, None, None]
            return x.permute(1, 0, 2, 3).reshape(c["kv"], -1, c["dim"])[:, :length]

        k, v = tokens(s["k_codes"], s["k_scales"]), tokens(s["v_codes"], s["v_scales"])
        for r in range(rows):
            seen = max(0, length - rows + r + 1)
            q = s["q"][starts[i] + r].double().view(c["kv"], group, c["dim"])
            score = torch.einsum("hgd,htd->hgt", q, k[:, :seen]) * s["scale"]
            if seen:
                lse = torch.logsumexp(score, 2)
                out = torch.einsum("hgt,htd->hgd", torch.exp(score - lse[:, :, None]), v[:, :seen])
            else:
                lse, out = torch.full((c["kv"], group), -math.inf, dtype=torch.float64, device=DEV), torch.zeros_like(q)
            outs.append(out.reshape(1, c["heads"], c["dim"]))
            lses.append(lse.reshape(1, c["heads"]))
    return dict(out=torch.cat(outs), lse=torch.cat(lses))
