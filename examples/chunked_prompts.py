"""Prompts that go into the cache a chunk at a time, with rotary positions, then decode steps behind them.

Each step gives every request some of its prompt's next tokens, as many as fit the step's rows, and runs one attention layer:

  fp8blk_gemv            q, k, v of the rows (FP8 block-scaled weights, f32 activations)
  fp8blk_kv_map          seq_lens, q_starts, slots, positions and block tables, on the device
  fp8blk_rope_table      the rows' cosines and sines, from their positions
  fp8blk_kv_append_rope  k rotated into the paged e4m3 cache, v beside it, q rotated in place
  fp8blk_kv_attn_chunk   the chunks' attention over the cache, their own tokens and those of earlier steps
  fp8blk_gemv            output projection

Then single tokens take the same way, with fp8blk_kv_attn for the attention.  Weights and hidden states are random; a real
engine runs the part between the map and the output projection once per layer, with one table for all of them.
Run: python examples/chunked_prompts.py
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from fp8_block_scaled_fp8blk_gb300 import ops  # noqa: E402
from verify_step import Cache, Model, linear  # noqa: E402


def layer(model: Model, cache: Cache, ctx_lens, new_lens, hidden, turns, attn_scale, ws, chunk: bool) -> dict:
    """One step's rows through the layer; what came in between is handed back too."""
    rows, d = hidden.shape[0], model.head_dim
    step = cache.map(ctx_lens, new_lens, rows)
    qkv = linear(model.qkv, hidden).view(rows, -1, d)
    before = qkv.clone()
    q, k, v = qkv.split([model.q_heads, model.kv_heads, model.kv_heads], dim=1)
    cos_sin = ops.fp8blk_rope_table(step.positions, turns, attn_scale)
    ops.fp8blk_kv_append_rope(k, v, step.slots, cos_sin, *cache.pools, q=q, q_out=q)
    args = (q, *cache.pools, cache.table, step.seq_lens, step.q_starts)
    scale = 1.0 / math.sqrt(d)
    attn = ops.fp8blk_kv_attn_chunk(*args, scale, ws) if chunk else ops.fp8blk_kv_attn(*args, 1, scale, ws)
    x = hidden + linear(model.out, attn.reshape(rows, model.q_heads * d))
    return dict(step=step, qkv=before, q=q, attn=attn, x=x, cos_sin=cos_sin, scale=scale, chunk=chunk)


def main(prompts=(150, 37, 260), rows: int = 128, decode: int = 2, seed: int = 0, keep=lambda cache, out: out) -> list:
    """The steps' results in turn; `keep` sees the cache after each."""
    model, n = Model(), len(prompts)
    gen = torch.Generator(device=model.device)
    gen.manual_seed(seed)
    cache = Cache(model, n_seqs=n, n_blocks=48, block_tokens=16, max_blocks=20)
    freqs, attn_scale = ops.rope_frequencies(model.head_dim, 10000.0, "ramp", factor=4.0, original_len=64.0, low=1.0, high=32.0)
    turns = ops.rope_turns(freqs, model.device)
    ws = ops.kv_attn_chunk_workspace(model.q_heads, model.kv_heads, model.head_dim, model.device)
    one = ops.kv_attn_workspace(n, 1, model.q_heads, model.kv_heads, model.head_dim, model.device)
    done, left, results = [0] * n, list(prompts), []

    def run(new, chunk):
        hidden = torch.randn((sum(new), model.hidden), device=model.device, generator=gen)
        ctx_lens, new_lens = (torch.tensor(x, dtype=torch.int32, device=model.device) for x in (done, new))
        results.append(keep(cache, layer(model, cache, ctx_lens, new_lens, hidden, turns, attn_scale, ws if chunk else one, chunk)))
        for i, x in enumerate(new):
            done[i] += x

    while any(left):
        room, new = rows, []
        for x in left:
            new.append(min(x, room))
            room -= new[-1]
        left = [a - b for a, b in zip(left, new)]
        run(new, True)
        print(f"step {len(results)}: rows {new}, tokens in the cache {done}")
    for _ in range(decode):
        run([1] * n, False)
        print(f"step {len(results)}: a token each, tokens in the cache {done}")
    if ops.fp8blk_device_status(clear=True):
        raise RuntimeError("a kernel reported a problem")
    return results


if __name__ == "__main__":
    main()
