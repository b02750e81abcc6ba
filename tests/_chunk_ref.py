"""Attention of a request's rows over a paged cache in 64 bits (numpy), for the tests of fp8blk_kv_attn_chunk."""
import numpy as np

import _step_ref as ref


def attn(q, k_codes, k_scales, v_codes, v_scales, table, lens, starts, scale):
    """out, lse, and what error bounds need, per (row, head): the largest scale * sum_d |q k_t| (peak), the tokens seen, the
    largest p_t |s_v(t)|; per output element sum_t p_t |v_t| (spread).  p is normalised."""
    rows, heads, dim = q.shape
    kv, block = k_codes.shape[1], k_codes.shape[2]
    group = heads // kv
    out, lse = np.zeros((rows, heads, dim)), np.full((rows, heads), -np.inf)
    peak, spread = np.zeros((rows, heads)), np.zeros((rows, heads, dim))
    seen_all, top = np.zeros((rows, heads)), np.zeros((rows, heads))
    for s in range(len(lens)):
        r, n = int(starts[s + 1] - starts[s]), int(lens[s])
        if r == 0 or n == 0:
            continue
        ids = table[s, : -(-n // block)]
        seen = np.arange(n)[None] <= (n - r + np.arange(r))[:, None]
        for g in range(kv):
            sv = np.repeat(np.abs(v_scales[ids, g].astype(np.float64)), block)[:n]
            k = (ref.E4M3[k_codes[ids, g]] * k_scales[ids, g, None, None].astype(np.float64)).reshape(-1, dim)[:n]
            v = (ref.E4M3[v_codes[ids, g]] * v_scales[ids, g, None, None].astype(np.float64)).reshape(-1, dim)[:n]
            for h in range(g * group, (g + 1) * group):
                x = q[starts[s]: starts[s] + r, h]
                a = np.where(seen, scale * (x @ k.T), -np.inf)
                m = a.max(1, keepdims=True)
                live = np.isfinite(m[:, 0])
                e = np.exp(a - np.where(live[:, None], m, 0.0))
                z = e.sum(1, keepdims=True)
                p = e / np.where(z > 0, z, 1.0)
                at = slice(int(starts[s]), int(starts[s]) + r)
                out[at, h], spread[at, h] = p @ v, p @ np.abs(v)
                lse[at, h] = np.where(live, (m + np.log(np.where(z > 0, z, 1.0)))[:, 0], -np.inf)
                peak[at, h] = np.where(seen, abs(scale) * (np.abs(x) @ np.abs(k).T), 0.0).max(1)
                seen_all[at, h], top[at, h] = seen.sum(1), (p * sv).max(1)
    return out, lse, peak, spread, seen_all, top


def tolerances(want, wlse, peak, spread, seen, top, dim, bf16):
    """Bounds on |out - want| and |lse - wlse|, from the arithmetic (see test_kv_chunk_gpu)."""
    u = (dim + 24) * 2.0 ** -24
    w = 2.0 ** -11 if bf16 else 2.0 ** -22
    sums = (seen / 16 + 32) * 2.0 ** -23
    out = (2 * u * peak + w + 2.0 ** -20 + sums)[:, :, None] * spread + (2.0 ** -30 * 448 * seen * top)[:, :, None]
    if bf16:
        out = out + 2.0 ** -8 * np.abs(want) + 1e-38
    return out, u * peak + 2.0 ** -20 + sums + 2.0 ** -23 * np.abs(np.where(np.isfinite(wlse), wlse, 0.0))
