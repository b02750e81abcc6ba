"""One speculative verify step around the library's calls, from hidden states to scored drafts.

A batch of requests, each with its cached context and up to eight new rows (the last accepted token and its drafts), goes
through one attention layer and the vocab head:

  fp8blk_gemv            q, k, v of each request's rows (FP8 block-scaled weights, f32 activations)
  fp8blk_kv_map          seq_lens, q_starts, slots and block tables, on the device
  fp8blk_kv_append       k, v into the paged e4m3 cache
  fp8blk_kv_attn         the rows' attention over it
  fp8blk_gemv            output projection
  fp8blk_gemv_argmax     vocab head: the greedy token and the logits of every row
  fp8blk_token_logprobs  each draft's log probability and rank, the entropy, and the likeliest alternatives

A draft is accepted while it is the greedy token of the row before it.  Then loop() runs steps in a row: rejected rows'
slots are written again, and a block that only they had reached stays their request's.  Weights are random; a real engine
runs the middle part once per layer.  Run: python examples/verify_step.py
"""
from __future__ import annotations

import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp8_block_scaled_fp8blk_gb300 import ops, synth  # noqa: E402


class Model:
    """One layer's projections and the head, as FP8 codes with a grid of power-of-two scales."""

    def __init__(self, hidden=512, q_heads=8, kv_heads=2, head_dim=64, vocab=2000, device="cuda:0"):
        self.hidden, self.q_heads, self.kv_heads, self.head_dim, self.vocab = hidden, q_heads, kv_heads, head_dim, vocab
        self.device = device

        def weight(rows, cols, seed):
            c = synth.fp8blk_case(rows, cols, 1, seed)
            scale = (c.scale_e8m0.astype(np.int32) - 9).astype(np.uint8)  # keep activations of order one
            return (torch.from_numpy(c.codes).to(device), torch.from_numpy(ops.fp8blk_scales_from_e8m0(scale)).to(device))

        self.qkv = weight((q_heads + 2 * kv_heads) * head_dim, hidden, 1)
        self.out = weight(hidden, q_heads * head_dim, 2)
        self.head = weight(vocab, hidden, 3)


class Cache:
    """A pool of blocks, the requests' tables over it, and the list of free blocks."""

    def __init__(self, model: Model, n_seqs: int, n_blocks: int, block_tokens: int, max_blocks: int):
        d, shape = model.device, (n_blocks, model.kv_heads, block_tokens, model.head_dim)
        self.block_tokens = block_tokens
        self.k_codes, self.v_codes = (torch.zeros(shape, dtype=torch.uint8, device=d) for _ in range(2))
        self.k_scales, self.v_scales = (torch.zeros(shape[:2], dtype=torch.float32, device=d) for _ in range(2))
        self.table = torch.full((n_seqs, max_blocks), -1, dtype=torch.int32, device=d)
        self.free_blocks = torch.arange(n_blocks, dtype=torch.int32, device=d)
        self.free_head = torch.zeros(1, dtype=torch.int32, device=d)
        self.held, self._spare = (torch.zeros(n_seqs, dtype=torch.int32, device=d) for _ in range(2))

    def map(self, ctx_lens, new_lens, max_tokens: int):
        """Blocks and slots for new tokens; blocks of rejected ones stay their request's for the next."""
        step = ops.fp8blk_kv_map(ctx_lens, new_lens, self.table, self.free_blocks, self.free_head, self.block_tokens, max_tokens,
                                 held=self.held, held_out=self._spare)
        self.free_head, self.held, self._spare = step.free_head, self._spare, self.held
        return step

    @property
    def pools(self):
        return self.k_codes, self.k_scales, self.v_codes, self.v_scales


def linear(weight, x):
    """x [rows, cols] through an FP8 weight, at most ops.MAX_M rows a call."""
    codes, scales = weight
    y = torch.empty((x.shape[0], codes.shape[0]), dtype=torch.float32, device=x.device)
    for r in range(0, x.shape[0], ops.MAX_M):
        ops.fp8blk_gemv(codes, scales, x[r: r + ops.MAX_M].contiguous(), y[r: r + ops.MAX_M])
    return y


def fill(model: Model, cache: Cache, lens: torch.Tensor, hidden: torch.Tensor) -> None:
    """Prompts: keys and values of all their tokens in one call."""
    step = cache.map(torch.zeros_like(lens), lens, hidden.shape[0])
    qkv = linear(model.qkv, hidden).view(hidden.shape[0], -1, model.head_dim)
    k, v = qkv[:, model.q_heads: model.q_heads + model.kv_heads], qkv[:, model.q_heads + model.kv_heads:]
    ops.fp8blk_kv_append(k, v, step.slots, *cache.pools)


def verify(model: Model, cache: Cache, ctx_lens, new_lens, hidden, drafts, ws, top=4):
    """One step: hidden [rows, hidden], drafts [rows] (the token each row is asked about; -1 = none)."""
    rows, d = hidden.shape[0], model.head_dim
    step = cache.map(ctx_lens, new_lens, rows)
    qkv = linear(model.qkv, hidden).view(rows, -1, d)
    q = qkv[:, : model.q_heads]
    k, v = qkv[:, model.q_heads: model.q_heads + model.kv_heads], qkv[:, model.q_heads + model.kv_heads:]
    ops.fp8blk_kv_append(k, v, step.slots, *cache.pools)
    attn = ops.fp8blk_kv_attn(q, *cache.pools, cache.table, step.seq_lens, step.q_starts, ops.MAX_M, 1.0 / math.sqrt(d), ws)
    x = hidden + linear(model.out, attn.reshape(rows, model.q_heads * d))
    logits = torch.empty((rows, model.vocab), dtype=torch.float32, device=model.device)
    tokens = torch.empty(rows, dtype=torch.int32, device=model.device)
    arg_ws = ops.argmax_workspace(ops.MAX_M, model.vocab, model.hidden, model.device)
    codes, scales = model.head
    for r in range(0, rows, ops.MAX_M):
        e = min(rows, r + ops.MAX_M)
        ops.fp8blk_gemv_argmax(codes, scales, x[r:e].contiguous(), arg_ws, tokens=tokens[r:e], logits=logits[r:e])
    return step, attn, logits, tokens, ops.fp8blk_token_logprobs(logits, drafts, top)


def main(seed: int = 0) -> dict:
    model = Model()
    gen = torch.Generator(device=model.device)
    gen.manual_seed(seed)
    lens = torch.tensor([70, 5, 33], dtype=torch.int32, device=model.device)
    cache = Cache(model, n_seqs=3, n_blocks=24, block_tokens=16, max_blocks=8)
    total = int(lens.sum())
    fill(model, cache, lens, torch.randn((total, model.hidden), device=model.device, generator=gen))

    new = torch.tensor([8, 3, 1], dtype=torch.int32, device=model.device)
    rows = int(new.sum())
    hidden = torch.randn((rows, model.hidden), device=model.device, generator=gen)
    drafts = torch.randint(0, model.vocab, (rows,), device=model.device, generator=gen, dtype=torch.int32)
    starts = torch.cumsum(new, 0).cpu().tolist()
    drafts[[s - 1 for s in starts]] = -1  # a request's last row has no draft after it
    ws = ops.kv_attn_workspace(3, ops.MAX_M, model.q_heads, model.kv_heads, model.head_dim, model.device)
    step, attn, logits, tokens, scores = verify(model, cache, lens, new, hidden, drafts, ws)

    accepted = (tokens == drafts).cpu().tolist()
    first = 0
    for s, end in enumerate(starts):
        n = 0
        while first + n < end - 1 and accepted[first + n]:
            n += 1
        draft = (f"log p of the first draft {float(scores.logprob[first]):.3f} (rank {int(scores.rank[first])}), "
                 if end - first > 1 else "")
        print(f"request {s}: {end - first - 1} drafts, {n} accepted, next token {int(tokens[first + n])}, "
              f"{draft}entropy {float(scores.entropy[first]):.3f}")
        first = end
    if ops.fp8blk_device_status(clear=True):
        raise RuntimeError("a kernel reported a problem")
    return dict(model=model, cache=cache, step=step, hidden=hidden, drafts=drafts, attn=attn, logits=logits, tokens=tokens,
                scores=scores, lens=lens, new=new)


def loop(steps: int = 6, seed: int = 1):
    """Verify steps in a row: each request's context grows by its accepted rows only, the rejected ones' slots are written
    again, and the host is asked nothing in between."""
    model, n = Model(), 3
    gen = torch.Generator(device=model.device)
    gen.manual_seed(seed)
    lens = torch.tensor([30, 47, 64], dtype=torch.int32, device=model.device)
    cache = Cache(model, n, n_blocks=40, block_tokens=16, max_blocks=10)
    fill(model, cache, lens, torch.randn((int(lens.sum()), model.hidden), device=model.device, generator=gen))
    new = torch.full((n,), ops.MAX_M, dtype=torch.int32, device=model.device)
    rows = n * ops.MAX_M
    ws = ops.kv_attn_workspace(n, ops.MAX_M, model.q_heads, model.kv_heads, model.head_dim, model.device)
    accepted = torch.zeros((steps, n), dtype=torch.int32, device=model.device)
    for i in range(steps):
        hidden = torch.randn((rows, model.hidden), device=model.device, generator=gen)
        drafts = torch.randint(0, model.vocab, (n, ops.MAX_M), device=model.device, generator=gen, dtype=torch.int32)
        drafts[:, -1] = -1  # the last row has no draft after it
        tokens = verify(model, cache, lens, new, hidden, drafts.flatten(), ws)[3].view(n, -1)
        drafts[:, 0] = torch.where(torch.rand(n, device=model.device, generator=gen) < 0.5, tokens[:, 0], drafts[:, 0])
        accepted[i] = 1 + torch.cumprod((tokens == drafts).int(), 1).sum(1).int()
        lens = lens + accepted[i]
    counts = accepted.cpu()
    print(f"{steps} steps of {n} x {ops.MAX_M} rows: {counts.tolist()} rows accepted, {cache.held.tolist()} blocks held, "
          f"{int(cache.free_head)} taken")
    if ops.fp8blk_device_status(clear=True):
        raise RuntimeError("a kernel reported a problem")
    return cache, lens, counts


if __name__ == "__main__":
    main()
    loop()
