"""The 8-bit operators together, as a decode loop uses them: a prompt is
appended, then verify steps (attention, argmax and walk, commit) run over the
cache they extend, with the log probabilities of what they emit; all against
the float64 definitions. And the same log probabilities beside the Q4_0 step."""

import numpy as np
import pytest
import torch

import oracle
import oracle.int8 as I8
import oracle.logprobs as OL
from _helpers import DEV, bf16_dev, i32_dev, logits_dev, need_gpu
from tree_verify_attention_gb300 import api
from tree_verify_attention_gb300 import workload as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def bf16_values(x):
    return W.bf16_bits_to_f32(W.f32_to_bf16_bits(x))


@pytest.mark.parametrize("cfg,steps,graph", [(W.TINY, 12, False), (W.TINY, 12, True),
                                             (W.SHORT, 4, False)],
                         ids=["tiny", "tiny_graph", "short"])
def test_chained_steps(cfg, steps, graph):
    hkv, d, n = cfg.n_kv_heads, cfg.head_dim, cfg.n_nodes
    cap = cfg.ctx_len + steps * n
    kf, vf = W.make_context(cfg)                       # float32 [Hkv, C, D]
    cache = api.Int8Cache(hkv, d, cap, device=DEV)
    cache.fill(torch.from_numpy(kf).to(DEV), torch.from_numpy(vf).to(DEV))
    hist = [bf16_values(kf), bf16_values(vf)]          # the rows as the cache takes them
    step = api.VerifyStep(n, cfg.n_q_heads, hkv, d, cfg.window, cap, cfg.vocab,
                          max_depth=cfg.max_depth, fmt="int8", top=4)
    bufs, g = None, None
    for i in range(steps):
        s = W.make_step(cfg, i)
        new = (bf16_dev(s.q), bf16_dev(s.k_tree), bf16_dev(s.v_tree), i32_dev(s.parent),
               i32_dev(s.tokens), logits_dev(s.logits))
        if not graph:
            step.run(cache, *new)
        else:
            if bufs is None:
                bufs = [t.clone() for t in new]
                end = cache.open_end.clone()
                step.run(cache, *bufs)                 # loads the kernels before the capture
                cache.open_end.copy_(end)
                torch.cuda.synchronize()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    step.run(cache, *bufs)
            for b, t in zip(bufs, new):
                b.copy_(t)
            g.replay()
        torch.cuda.synchronize()
        C = hist[0].shape[1]
        kt, vt = W.bf16_bits_to_f32(s.k_tree), W.bf16_bits_to_f32(s.v_tree)
        out, lse = oracle.attention.tree_verify_attention_by_head(
            W.bf16_bits_to_f32(s.q), I8.cached_values(hist[0]), I8.cached_values(hist[1]), kt, vt,
            s.parent, C, cfg.window)
        logits = (W.bf16_bits_to_f32(s.logits) if s.logits.dtype == np.uint16 else s.logits)
        argmax = oracle.accept.node_argmax(logits)
        path, emitted = oracle.accept.greedy_walk(s.parent, s.tokens, argmax)
        L = len(path)
        assert int(step.status) == 0 and int(step.accept_len) == L
        assert step.argmax.cpu().numpy().tolist() == argmax.tolist()
        assert step.path.cpu().numpy()[:L].tolist() == path.tolist()
        assert step.out_tokens.cpu().numpy()[:L].tolist() == emitted.tolist()
        # weights rounded to binary16 and scores of float32 sums of 256 products
        # at most: see test_gpu_int8_attn.py; the values here are unit normals
        assert np.abs(step.out.double().cpu().numpy() - out).max() < 4e-3
        assert np.abs(step.lse.double().cpu().numpy() - lse).max() < 1e-3
        lp, ent, ids, tlp = OL.token_logprobs(logits, argmax, 4)
        assert np.array_equal(step.top_ids.cpu().numpy(), ids)
        assert np.abs(step.logprob.cpu().numpy() - lp).max() < 1e-4
        assert np.abs(step.entropy.cpu().numpy() - ent).max() < 1e-3
        assert np.abs(step.top_logprobs.cpu().numpy() - tlp).max() < 1e-4
        hist = [np.concatenate([h, t[path].transpose(1, 0, 2)], axis=1)
                for h, t in zip(hist, (kt, vt))]
        assert int(cache.ctx_len) == C + L
        nb = (C + L) // 64
        codes, scale = I8.encode_blocks(hist[0])
        assert np.array_equal(I8.unpack_k(cache.k.cpu().numpy())[:, :nb], codes)
        assert np.array_equal(cache.k_scale.cpu().numpy()[:, :nb], scale)


def test_a_single_node_step_is_plain_decode():
    """Budget 0: one query, its own row appended, over 130 steps (two blocks
    close on the way)."""
    hq, hkv, d = 6, 2, 128
    rng = np.random.default_rng(3)
    cache = api.Int8Cache(hkv, d, 200, device=DEV)
    ws = api.workspace(api.int8_attn_workspace_bytes(1, hq, hkv, d, 0, 200))
    par, one = i32_dev([-1]), i32_dev([1])
    zero = i32_dev([0])
    rows = [np.zeros((hkv, 0, d)), np.zeros((hkv, 0, d))]
    out, lse = torch.empty(1, hq, d, device=DEV), torch.empty(1, hq, device=DEV)
    for i in range(130):
        q, k, v = (W.f32_to_bf16_bits(rng.standard_normal((1, h, d))) for h in (hq, hkv, hkv))
        api.tree_verify_attn(cache, bf16_dev(q), bf16_dev(k), bf16_dev(v), par, 0, 1, out, lse, ws)
        api.kv_commit(cache, one, zero, bf16_dev(k), bf16_dev(v))
        if i % 9 == 0 or i in (63, 64, 65, 127, 128, 129):
            want, wlse = oracle.attention.tree_verify_attention_by_head(
                W.bf16_bits_to_f32(q), I8.cached_values(rows[0]), I8.cached_values(rows[1]),
                W.bf16_bits_to_f32(k), W.bf16_bits_to_f32(v), np.array([-1]), i, 0)
            assert np.abs(out.double().cpu().numpy() - want).max() < 4e-3
            assert np.abs(lse.double().cpu().numpy() - wlse).max() < 1e-3
        rows = [np.concatenate([r, W.bf16_bits_to_f32(x).transpose(1, 0, 2)], axis=1)
                for r, x in zip(rows, (k, v))]
    assert int(cache.ctx_len) == 130 and int(cache.status) == 0


def test_log_probabilities_beside_the_q4_0_step():
    cfg = W.TINY
    s = W.make_step(cfg)
    kf, vf = W.make_context(cfg)
    cap = cfg.ctx_len + cfg.n_nodes
    cache = api.Q4Cache(cfg.n_kv_heads, cfg.head_dim, cap)
    cache.fill(torch.from_numpy(kf).to(DEV), torch.from_numpy(vf).to(DEV))
    step = api.VerifyStep(cfg.n_nodes, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim, cfg.window,
                          cap, cfg.vocab, max_depth=cfg.max_depth, top=0)
    step.run(cache, bf16_dev(s.q), bf16_dev(s.k_tree), bf16_dev(s.v_tree), i32_dev(s.parent),
             i32_dev(s.tokens), logits_dev(s.logits))
    lp, ent, _, _ = OL.token_logprobs(s.logits, oracle.accept.node_argmax(s.logits), 1)
    assert int(step.status) == 0
    assert np.abs(step.logprob.cpu().numpy() - lp).max() < 1e-4
    assert np.abs(step.entropy.cpu().numpy() - ent).max() < 1e-3


def test_the_step_refuses_what_it_is_not_planned_for():
    with pytest.raises(api.DfvError, match="pipelined"):
        api.VerifyStep(9, 4, 1, 64, 0, 300, 1000, fmt="int8", pipelined=True)
    with pytest.raises(api.DfvError, match="unknown cache format"):
        api.VerifyStep(9, 4, 1, 64, 0, 300, 1000, fmt="int4")
    step = api.VerifyStep(9, 4, 1, 64, 0, 300, 1000, fmt="int8")
    other = api.VerifyStep(9, 4, 1, 64, 0, 300, 1000)
    with pytest.raises(api.DfvError, match="another kind"):
        step.run(api.Q4Cache(1, 64, 300), *[None] * 6)
    with pytest.raises(api.DfvError, match="another kind"):
        other.run(api.Int8Cache(1, 64, 300), *[None] * 6)
    with pytest.raises(api.DfvError, match="capacity"):
        step.run(api.Int8Cache(1, 64, 301), *[None] * 6)
