"""GPU test of the example that runs the cache, attention and scoring calls together (examples/verify_step.py): its
attention and scores against the plain 64-bit restatements, from the cache that its own calls filled."""
import importlib.util
import os

import numpy as np
import pytest

import _step_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_verify_step_example():
    spec = importlib.util.spec_from_file_location("verify_step", os.path.join(ROOT, "examples", "verify_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.main()
    model, cache, step = r["model"], r["cache"], r["step"]
    host = [t.cpu().numpy() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    lens, starts = step.seq_lens.cpu().numpy(), step.q_starts.cpu().numpy()
    assert lens.tolist() == [78, 8, 34] and starts.tolist() == [0, 8, 11, 12]
    qkv = m.linear(model.qkv, r["hidden"]).view(12, -1, model.head_dim)
    q = qkv[:, : model.q_heads].cpu().numpy().astype(np.float64)
    want, _, peak, spread = ref.kv_attn(q, *host, cache.table.cpu().numpy(), lens, starts, model.head_dim ** -0.5)
    u = 2.0 ** -16 + (model.head_dim + 16) * 2.0 ** -24
    tol = (2 * u * peak[:, :, None] + 2.0 ** -16 + 2.0 ** -19) * spread
    assert (np.abs(r["attn"].cpu().numpy() - want) <= tol).all()
    logprob, rank, entropy, ids, tops = ref.token_logprobs(r["logits"].cpu().numpy().astype(np.float64), r["drafts"].cpu().numpy(), 4)
    s = r["scores"]
    assert np.array_equal(s.rank.cpu().numpy(), rank) and np.array_equal(s.top_ids.cpu().numpy(), ids)
    assert np.array_equal(s.top_ids[:, 0].cpu().numpy(), r["tokens"].cpu().numpy())
    span = 2.0 ** -18 * (1 + np.abs(r["logits"].cpu().numpy()).max(1))
    have = rank >= 0
    assert (np.abs(s.logprob.cpu().numpy() - logprob)[have] <= span[have]).all()
    assert (np.abs(s.entropy.cpu().numpy() - entropy) <= 3 * span).all()
    # The cache holds what was appended: every used block's scale is a power of two that its largest code needs.
    used = cache.table.cpu().numpy()
    for k in (1, 3):
        m2, _ = np.frexp(host[k][used[used >= 0]])
        assert (m2 == 0.5).all()
