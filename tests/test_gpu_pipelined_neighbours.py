"""Pipelined verify steps with the library's other kernels before them in the
stream: a step reads its inputs before it waits for the kernel before it, so
that kernel must not have let the step start before what wrote the inputs has
completed. And pipelined steps with log probabilities, which stand between the
steps of a chain, against plain launches."""

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


NAMES = ("out", "lse", "argmax", "accept_len", "path", "out_tokens", "status", "logprob",
         "entropy", "top_ids", "top_logprobs")


@pytest.mark.parametrize("fmt", ["q4_0", "f16"])
@pytest.mark.parametrize("cfg", [W.TINY, W.SHORT], ids=lambda c: c.name)
def test_chain_with_log_probabilities_equals_plain(cfg, fmt):
    n = 10
    pool = [W.make_step(cfg, i) for i in range(5)]
    ins = [(bf16_dev(s.q), bf16_dev(s.k_tree), bf16_dev(s.v_tree), i32_dev(s.parent),
            i32_dev(s.tokens), logits_dev(s.logits)) for s in pool]
    cap = cfg.ctx_len + (n + 2) * cfg.n_nodes
    kf, vf = (torch.from_numpy(x).to(DEV) for x in W.make_context(cfg))

    def chain(pipelined):
        cache = api.KVCache(cfg.n_kv_heads, cfg.head_dim, cap, fmt=fmt)
        cache.fill(kf, vf)
        step = api.VerifyStep(cfg.n_nodes, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim, cfg.window,
                              cap, cfg.vocab, max_depth=cfg.max_depth, pipelined=pipelined, top=4)
        kept = []
        torch.cuda.synchronize()
        for i in range(n):                     # no synchronisation on the host in between
            step.run(cache, *ins[i % 5])
            kept.append([getattr(step, k).clone() for k in NAMES])
        # and with nothing but the log probabilities between two steps
        for i in range(n):
            step.run(cache, *ins[i % 5])
        kept.append([getattr(step, k).clone() for k in NAMES])
        torch.cuda.synchronize()
        return cache, kept

    cap += n * cfg.n_nodes
    c0, k0 = chain(False)
    c1, k1 = chain(True)
    for a, b in zip(k0, k1):
        for name, x, y in zip(NAMES, a, b):
            assert torch.equal(x.view(torch.int32), y.view(torch.int32)), name
    assert torch.equal(c0.k, c1.k) and torch.equal(c0.v, c1.v)
    assert int(c0.ctx_len) == int(c1.ctx_len)
    s = pool[(n - 1) % 5]
    logits = W.bf16_bits_to_f32(s.logits) if s.logits.dtype == np.uint16 else s.logits
    argmax = oracle.accept.node_argmax(logits)
    lp, ent, ids, _ = OL.token_logprobs(logits, argmax, 4)
    got = dict(zip(NAMES, (x.cpu().numpy() for x in k1[n - 1])))
    assert int(got["status"][0]) == 0 and np.array_equal(got["top_ids"], ids)
    assert np.abs(got["logprob"] - lp).max() < 1e-4 and np.abs(got["entropy"] - ent).max() < 1e-3


@pytest.mark.parametrize("between", ["logprobs", "append", "long_append", "commit", "read",
                                     "attention"])
def test_inputs_written_by_the_kernel_before_the_one_before(between):
    """The draft's tokens are the alternatives of a row of 2^26 logits, still
    being read when the small kernel between is launched."""
    n, hq, hkv, d, vocab, cap = 9, 4, 1, 64, 1000, 400
    tok = torch.randperm(vocab, generator=torch.Generator().manual_seed(5))[:n]
    big = torch.zeros(1, 1 << 26, device=DEV)
    big[0, tok.to(DEV)] = torch.arange(n, 0, -1, device=DEV, dtype=torch.float32)
    logits = torch.zeros(n, vocab, device=DEV)
    logits[torch.arange(n - 1), tok[1:]] = 5.0        # node i asks for node i + 1's token
    q, tk, tv = (torch.randn(n, h, d, device=DEV).to(torch.bfloat16) for h in (hq, hkv, hkv))
    parent = torch.arange(-1, n - 1, dtype=torch.int32, device=DEV)
    cache = api.Q4Cache(hkv, d, cap)
    cache.fill(torch.randn(hkv, 100, d, device=DEV), torch.randn(hkv, 100, d, device=DEV))
    step = api.VerifyStep(n, hq, hkv, d, 0, cap, vocab, pipelined=True)
    tokens = torch.empty(1, n, dtype=torch.int32, device=DEV)
    # what the kernels between work on
    other = api.Int8Cache(8, 256, 8192)
    rows = torch.randn(4000, 8, 256, device=DEV).to(torch.bfloat16)
    other.append(rows[:130], rows[:130])
    out = torch.empty(10, 8, 256, device=DEV), torch.empty(10, 8, 256, device=DEV)
    q8, par = rows[:1].contiguous(), parent[:1]
    o8 = torch.empty(1, 8, 256, device=DEV)
    ws = api.workspace(api.int8_attn_workspace_bytes(1, 8, 8, 256, 0, 8192))
    one, zero = i32_dev([1]), i32_dev([0])
    lp = torch.empty(2, device=DEV)
    some = torch.zeros(2, dtype=torch.int32, device=DEV)
    run = {"logprobs": lambda: api.token_logprobs(logits[:2], some, lp),
           "append": lambda: other.append(rows[:3], rows[:3], at=128),
           "long_append": lambda: other.append(rows, rows, at=0),
           "commit": lambda: api.kv_commit(other, one, zero, rows[:1], rows[:1]),
           "read": lambda: other.read(5, 10, *out),
           "attention": lambda: api.tree_verify_attn(other, q8, rows[:1], rows[:1], par, 0, 1, o8,
                                                     None, ws)}[between]
    for _ in range(6):
        cache.ctx_len.fill_(100)
        tokens.fill_(-1)
        step.accept_len.zero_()
        torch.cuda.synchronize()
        api.token_logprobs(big, None, None, None, tokens)
        run()
        step.run(cache, q, tk, tv, parent, tokens.view(n), logits)
        torch.cuda.synchronize()
        assert tokens[0].tolist() == tok.tolist()
        assert int(step.accept_len) == n and int(step.status) == 0
        assert step.path.tolist() == list(range(n))
    assert int(other.status) == 0
