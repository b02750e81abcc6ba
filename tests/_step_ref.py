"""Plain 64-bit restatements (numpy, loops) of the paged-cache and scoring calls, for the GPU tests.

Nothing here uses the package: codes are decoded by a table built from the
e4m3 bit fields and encoded by a search for the nearest table entry.
"""
import math

import numpy as np


def e4m3_table() -> np.ndarray:
    out = np.empty(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        v = math.nan if (e, f) == (15, 7) else math.ldexp(f, -9) if e == 0 else math.ldexp(8 + f, e - 10)
        out[b] = -v if b & 128 else v
    return out


E4M3 = e4m3_table()
_GRID = E4M3[:127]


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Nearest code, halves to the even one; beyond 448 the largest; what is not finite the NaN code (sign not kept)."""
    x = np.asarray(x, dtype=np.float64)
    good = np.isfinite(x)
    a = np.minimum(np.abs(np.where(good, x, 0.0)), 448.0)
    hi = np.clip(np.searchsorted(_GRID, a), 1, 126)
    lo = hi - 1
    down, up = a - _GRID[lo], _GRID[hi] - a
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code = code | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(good, code, np.uint8(0x7F)).astype(np.uint8)


def same_codes(a: np.ndarray, b: np.ndarray) -> bool:
    """Equal codes; the two NaN codes count as one."""
    nan_a, nan_b = (a & 0x7F) == 0x7F, (b & 0x7F) == 0x7F
    return bool(np.array_equal(nan_a, nan_b) and np.array_equal(a[~nan_a], b[~nan_b]))


def pow2_scale(amax: float) -> float:
    """Smallest power of two s >= 2^-126 with amax <= 448 s."""
    s = 2.0 ** -126
    if amax > 448.0 * s:
        s = 2.0 ** math.ceil(math.log2(amax / 448.0) - 1e-9)
        while amax > 448.0 * s:
            s *= 2.0
        while s > 2.0 ** -126 and amax <= 448.0 * (s / 2.0):
            s /= 2.0
    return s


def kv_map(ctx, new, table, free, head, block, max_tokens):
    """(table, seq_lens, q_starts, slots, positions, head, exhausted, bad)."""
    n, width = table.shape
    table = table.copy()
    slots, positions = np.full(max_tokens, -1, np.int64), np.full(max_tokens, -1, np.int32)
    lens, starts = np.zeros(n, np.int32), np.zeros(n + 1, np.int32)
    exhausted, bad, at = False, head < 0, 0
    head = max(head, 0)
    for r in range(n):
        c, f = max(int(ctx[r]), 0), max(int(new[r]), 0)
        bad |= ctx[r] < 0 or new[r] < 0 or -(-(c + f) // block) > width
        lens[r], starts[r] = c + f, min(at, max_tokens)
        for b in range(min(-(-c // block), width), min(-(-(c + f) // block), width)):
            table[r, b] = free[head] if head < len(free) else -1
            exhausted |= head >= len(free)
            head += 1
        for p in range(c, c + f):
            if at < max_tokens:
                positions[at] = p
                if p // block < width and table[r, p // block] >= 0:
                    slots[at] = int(table[r, p // block]) * block + p % block
            else:
                bad = True
            at += 1
    starts[n] = min(at, max_tokens)
    return table, lens, starts, slots, positions, min(head, max(len(free), 0)), exhausted, bad


def kv_append(x, slots, codes, scales, block):
    """One pool after the call (x [n, heads, dim] in 64 bits)."""
    codes, scales = codes.copy(), scales.astype(np.float64)
    n, t = len(slots), 0
    while t < n:
        if slots[t] < 0:
            t += 1
            continue
        page, off = int(slots[t]) // block, int(slots[t]) % block
        run = 1
        while t + run < n and off + run < block and slots[t + run] == slots[t] + run:
            run += 1
        for h in range(x.shape[1]):
            rows = x[t: t + run, h]
            fin = np.abs(rows[np.isfinite(rows)])
            s = pow2_scale(float(fin.max()) if fin.size else 0.0)
            if off:
                old = scales[page, h]
                if old < s:
                    codes[page, h, :off] = e4m3_encode(E4M3[codes[page, h, :off]] * (old / s))
                s = max(s, old)
            codes[page, h, off: off + run] = e4m3_encode(rows / s)
            scales[page, h] = s
        t += run
    return codes, scales


def kv_attn(q, k_codes, k_scales, v_codes, v_scales, table, lens, starts, scale):
    """out, lse, and what error bounds need: per (row, head) the largest
    scale * sum_d |q k_t|, and per output element sum_t p_t |v_t|."""
    rows, heads, dim = q.shape
    kv, block = k_codes.shape[1], k_codes.shape[2]
    group = heads // kv
    out, lse = np.zeros((rows, heads, dim)), np.full((rows, heads), -np.inf)
    peak, spread = np.zeros((rows, heads)), np.zeros((rows, heads, dim))
    for s in range(len(lens)):
        r = starts[s + 1] - starts[s]
        for i in range(r):
            seen = lens[s] - r + i + 1
            if seen <= 0:
                continue
            ids = table[s, : -(-seen // block)]
            for h in range(heads):
                g = h // group
                k = (E4M3[k_codes[ids, g]] * k_scales[ids, g, None, None].astype(np.float64)).reshape(-1, dim)[:seen]
                v = (E4M3[v_codes[ids, g]] * v_scales[ids, g, None, None].astype(np.float64)).reshape(-1, dim)[:seen]
                row = starts[s] + i
                a = scale * (k @ q[row, h])
                m = a.max()
                e = np.exp(a - m)
                z = e.sum()
                out[row, h], lse[row, h] = (e / z) @ v, m + math.log(z)
                peak[row, h] = abs(scale) * (np.abs(k) @ np.abs(q[row, h])).max()
                spread[row, h] = (e / z) @ np.abs(v)
    return out, lse, peak, spread


def token_logprobs(x, targets, top):
    """logprob, rank, entropy, ids, top logprobs; x [n, vocab] in 64 bits."""
    n, vocab = x.shape
    logprob, rank, entropy = np.full(n, np.nan), np.full(n, -1, np.int32), np.full(n, np.nan)
    ids, tops = np.zeros((n, top), np.int32), np.full((n, top), np.nan)
    for i in range(n):
        row = x[i]
        key = np.where(np.isnan(row), -np.inf, row)
        order = np.lexsort((np.arange(vocab), np.isnan(row), -key))
        ids[i] = order[:top]
        if 0 <= targets[i] < vocab:
            rank[i] = int(np.nonzero(order == targets[i])[0][0])
        if np.isnan(row).any() or np.isposinf(row).any() or not np.isfinite(row).any():
            continue
        m = row.max()
        z = np.exp(row - m).sum()
        logp = row - m - math.log(z)
        p = np.exp(logp)
        entropy[i] = -(p[p > 0] * logp[p > 0]).sum()
        tops[i] = logp[ids[i]]
        if 0 <= targets[i] < vocab:
            logprob[i] = logp[targets[i]]
    return logprob, rank, entropy, ids, tops
