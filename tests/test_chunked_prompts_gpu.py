"""The rotary positions, the rotating append and the chunks' attention together: examples/chunked_prompts.py against a
64-bit restatement of each step, from the step's own inputs."""
import os
import sys

import numpy as np
import pytest
import torch

import _chunk_ref as cref
import _rope_ref as rref
import _step_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from fp8_block_scaled_fp8blk_gb300 import ops as o
    o.fp8blk_device_status(clear=True)
    yield o
    assert o.fp8blk_device_status(clear=True) == 0


def host(t):
    return t.cpu().numpy()


def snapshot(cache, out):
    out["pools"] = [host(t).copy() for t in cache.pools]
    out["table"] = host(cache.table).copy()
    return out


@pytest.mark.parametrize("prompts,rows", [((150, 37, 260), 128), ((9, 300), 309), ((1, 1, 2), 3)])
def test_steps(ops, prompts, rows):
    import chunked_prompts
    steps = chunked_prompts.main(prompts, rows, decode=2, keep=snapshot)
    assert [s["chunk"] for s in steps] == [True] * (len(steps) - 2) + [False] * 2
    heads, dim = steps[0]["q"].shape[1:]
    kv = steps[0]["pools"][0].shape[1]
    freqs, scale = rref.frequencies(dim, 10000.0, "ramp", 4.0, 64.0, 1.0, 32.0)
    keys = {}  # (request, position) -> rotated key in 64 bits, and the size of its products
    done = [0] * len(prompts)
    for n, s in enumerate(steps):
        starts, lens, pos = (host(t) for t in (s["step"].q_starts, s["step"].seq_lens, s["step"].positions))
        x = host(s["qkv"]).astype(np.float64)
        # Positions go on where the request's last chunk ended; q and k turn by them.
        want_pos = np.concatenate([np.arange(done[r], done[r] + starts[r + 1] - starts[r]) for r in range(len(prompts))])
        assert np.array_equal(pos[: len(want_pos)], want_pos)
        angle = want_pos[:, None] * freqs[None]
        cos, sin = np.cos(angle) * scale, np.sin(angle) * scale
        turned, size = rref.rotate(x, cos, sin, False, 0)
        q = host(s["q"]).astype(np.float64)
        # Cosines and sines to 2^-22 of the table's scale, two products and a sum in f32.
        tol = 2.0 ** -21 * (size + np.abs(scale) * np.abs(x).max(2, keepdims=True))
        assert (np.abs(q - turned[:, :heads]) <= tol[:, :heads]).all()
        # Attention of the rows the step holds, over what the cache then held.
        kc, ks, vc, vs = s["pools"]
        want, wlse, peak, spread, seen, top = cref.attn(q, kc, ks, vc, vs, s["table"], lens, starts, s["scale"])
        if s["chunk"]:
            bound, _ = cref.tolerances(want, wlse, peak, spread, seen, top, dim, False)
        else:  # fp8blk_kv_attn's, which keeps 2^-16 of a score
            u = 2.0 ** -16 + (dim + 16) * 2.0 ** -24
            bound = (2 * u * peak[:, :, None] + 2.0 ** -16 + 2.0 ** -19) * spread
        assert (np.abs(host(s["attn"]).astype(np.float64) - want) <= bound).all()
        # What the cache holds of each key so far: rounded to e4m3 once (2^-4 of it), and in the subnormals, 2^-10 of the
        # scale, whenever its block's scale grew.
        for r in range(len(prompts)):
            for i in range(starts[r], starts[r + 1]):
                keys[r, int(want_pos[i])] = turned[i, heads: heads + kv]
            done[r] += int(starts[r + 1] - starts[r])
            assert done[r] == lens[r]
        block = kc.shape[2]
        for (r, p), k in keys.items():
            b = s["table"][r, p // block]
            held = ref.E4M3[kc[b, :, p % block]] * ks[b].astype(np.float64)[:, None]
            assert (np.abs(held - k) <= 2.0 ** -4 * np.abs(k) * (1 + 2.0 ** -10) + ks[b][:, None] * ((n + 1) * 2.0 ** -10) + 1e-6).all()
    assert done == [p + 2 for p in prompts]


def test_two_graphs_share_a_workspace(ops):
    """A layer's calls in two graphs over one workspace, replayed in turn, give what the calls gave alone."""
    import chunked_prompts
    from verify_step import Cache, Model
    model = Model()
    gen = torch.Generator(device=model.device)
    gen.manual_seed(3)
    ws = ops.kv_attn_chunk_workspace(model.q_heads, model.kv_heads, model.head_dim, model.device)
    turns = ops.rope_turns(ops.rope_frequencies(model.head_dim, 10000.0)[0], model.device)
    lens = [torch.tensor(x, dtype=torch.int32, device=model.device) for x in ([60, 200, 3], [250, 1, 12])]
    hidden = [torch.randn((263, model.hidden), device=model.device, generator=gen) for _ in lens]
    zero = torch.zeros(3, dtype=torch.int32, device=model.device)

    def step(i):
        cache = Cache(model, 3, 48, 16, 20)
        return chunked_prompts.layer(model, cache, zero, lens[i], hidden[i], turns, 1.0, ws, True)["attn"]

    alone = [step(i).clone() for i in range(2)]
    graphs, outs = [], []
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(i))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for a, b in zip(alone, outs):
            assert torch.equal(a, b)
