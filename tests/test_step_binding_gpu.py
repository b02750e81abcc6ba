"""The binding refuses a tensor that is not on the call's device, before anything is launched: each argument of each call
of the step in turn is a host tensor among device tensors."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ops():
    from fp8_block_scaled_fp8blk_gb300 import ops as o
    yield o
    torch.cuda.synchronize()
    assert o.fp8blk_device_status(clear=True) == 0


def i32(*values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def refuses_host_tensors(call, args, more=()):
    """`args` are positional tensors (None: left out of the test), `more` what follows them."""
    for i, t in enumerate(args):
        if isinstance(t, torch.Tensor):
            with pytest.raises(ValueError):
                call(*args[:i], t.cpu(), *args[i + 1:], *more)
        elif isinstance(t, tuple):
            for j in range(len(t)):
                wrong = type(t)(*[x.cpu() if j == k else x for k, x in enumerate(t)])
                with pytest.raises(ValueError):
                    call(*args[:i], wrong, *args[i + 1:], *more)


def cache():
    kc = torch.zeros((4, 2, 16, 32), dtype=torch.uint8, device=DEV)
    ks = torch.zeros((4, 2), device=DEV)
    return kc, ks, kc.clone(), ks.clone()


def test_kv_map(ops):
    out = ops.kv_map_buffers(2, 8, DEV)
    table = torch.full((2, 2), -1, dtype=torch.int32, device=DEV)
    args = (i32(0, 0), i32(3, 2), table, i32(0, 1, 2, 3), i32(0))
    refuses_host_tensors(lambda a, b, c, d, e, o: ops.fp8blk_kv_map(a, b, c, d, e, 16, 8, out=o), args + (out,))
    assert int(table.max()) == -1


def test_kv_append(ops):
    x = torch.ones((3, 2, 32), device=DEV)
    c = cache()
    refuses_host_tensors(ops.fp8blk_kv_append, (x, x.clone(), torch.arange(3, device=DEV)) + c)
    assert int(c[0].max()) == 0


def test_kv_attn(ops):
    q = torch.ones((1, 4, 32), device=DEV)
    ws, out, lse = ops.kv_attn_workspace(1, 1, 4, 2, 32, DEV), torch.full_like(q, 3.0), torch.zeros((1, 4), device=DEV)
    args = (q,) + cache() + (i32(0).view(1, 1), i32(5), i32(0, 1), ws, out, lse)
    refuses_host_tensors(lambda *a: ops.fp8blk_kv_attn(*a[:8], 1, 1.0, a[8], out=a[9], lse=a[10]), args)
    with pytest.raises(ValueError):  # a workspace with holes in it
        ops.fp8blk_kv_attn(*args[:8], 1, 1.0, torch.zeros((ws.numel(), 2), dtype=torch.uint8, device=DEV)[:, 0], out=out)
    torch.cuda.synchronize()
    assert (out == 3).all()


def test_token_logprobs(ops):
    x = torch.zeros((3, 50), device=DEV)
    out = ops.token_logprobs_buffers(3, 2, DEV)
    refuses_host_tensors(lambda a, t, o: ops.fp8blk_token_logprobs(a, t, 2, out=o), (x, i32(0, 1, 2), out))


def test_gemv_and_experts(ops):
    from _helpers import scales_dev, to_dev
    from fp8_block_scaled_fp8blk_gb300 import synth
    c = synth.fp8blk_case(256, 256, 1, seed=1)
    w, s, x = to_dev(c.codes), scales_dev(c.scale_e8m0), to_dev(c.x)
    y = torch.full((1, 256), 3.0, device=DEV)
    refuses_host_tensors(ops.fp8blk_gemv, (w, s, x, y))
    ws, tok = ops.argmax_workspace(1, 256, 256, DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    refuses_host_tensors(ops.fp8blk_gemv_argmax, (w, s, x, ws, tok, y))
    refuses_host_tensors(ops.fp8blk_gemv_argmax_noalloc, (w, s, x, tok, y))
    refuses_host_tensors(ops.fp8blk_bf16_gemv, (torch.zeros((256, 256), dtype=torch.bfloat16, device=DEV), x, y))
    e = synth.nvfp4_case(2, 128, 512, 1, seed=2)
    codes, scales, g, ex = to_dev(e.codes), to_dev(e.scales), to_dev(e.gscale), to_dev(e.x)
    ye = torch.full((1, 128), 3.0, device=DEV)
    refuses_host_tensors(ops.nvfp4_expert_gemv, (codes, scales, g, i32(0), ex, ye))
    refuses_host_tensors(ops.mxfp4_expert_gemv, (codes, scales, i32(0), ex, ye))
    scratch = torch.zeros((128, 512), dtype=torch.int16, device=DEV)
    refuses_host_tensors(lambda a, b, o: ops.nvfp4_expert_dequant(a, b, e.gscale, 0, out=o), (codes, scales, scratch))
    refuses_host_tensors(lambda a, b, v, t, o: ops.nvfp4_expert_dequant_gemv(a, b, e.gscale, [0], v, t, y=o),
                         (codes, scales, ex, scratch, ye))
    torch.cuda.synchronize()
    assert (y == 3).all() and (ye == 3).all()


def test_pinned_host_memory_is_taken(ops):
    """The device reaches it: a token written straight to the host."""
    x = torch.randn((2, 1000), device=DEV)
    out = ops.token_logprobs_buffers(2, 1, DEV)
    pinned = out._replace(top_ids=torch.zeros((2, 1), dtype=torch.int32).pin_memory())
    ops.fp8blk_token_logprobs(x, i32(1, 2), 1, out=pinned)
    torch.cuda.synchronize()
    assert torch.equal(pinned.top_ids[:, 0], x.argmax(1).int().cpu())
