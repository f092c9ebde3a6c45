"""Log probabilities of a step whose logits come in another shape than
[N, vocab] (the steps over Q4_0 and F16 caches take any with as many)."""

import numpy as np
import pytest
import torch

import oracle
import oracle.logprobs as OL
from _helpers import DEV, bf16_dev, i32_dev, logits_dev, need_gpu
from tree_verify_attention_gb300 import api
from tree_verify_attention_gb300 import workload as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("fmt", ["q4_0", "f16"])
@pytest.mark.parametrize("shape", ["flat", "batched"])
def test_logits_of_another_shape(shape, fmt):
    cfg = W.TINY
    s = W.make_step(cfg)
    cap = cfg.ctx_len + cfg.n_nodes
    cache = api.KVCache(cfg.n_kv_heads, cfg.head_dim, cap, fmt=fmt)
    cache.fill(*(torch.from_numpy(x).to(DEV) for x in W.make_context(cfg)))
    step = api.VerifyStep(cfg.n_nodes, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim, cfg.window,
                          cap, cfg.vocab, max_depth=cfg.max_depth, top=3, fmt=fmt)
    x = logits_dev(s.logits)
    x = x.view(-1) if shape == "flat" else x[None]
    step.run(cache, bf16_dev(s.q), bf16_dev(s.k_tree), bf16_dev(s.v_tree), i32_dev(s.parent),
             i32_dev(s.tokens), x)
    logits = W.bf16_bits_to_f32(s.logits) if s.logits.dtype == np.uint16 else s.logits
    lp, ent, ids, _ = OL.token_logprobs(logits, oracle.accept.node_argmax(logits), 3)
    assert int(step.status) == 0 and np.array_equal(step.top_ids.cpu().numpy(), ids)
    assert np.abs(step.logprob.cpu().numpy() - lp).max() < 1e-4
    assert np.abs(step.entropy.cpu().numpy() - ent).max() < 1e-3
