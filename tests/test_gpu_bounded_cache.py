"""The operators around a step as they are used together: a projection's rows
normed and rotated to the tree's positions, a step that draws, the weights that
the cached keys received, and the rows that received the most moved to the other
of two caches, over and over; every part against float64 (the tolerances of each
operator's own tests), then replayed from a graph and on two streams at once."""

import math

import numpy as np
import pytest
import torch

import oracle
import oracle.encode as OE
import oracle.eviction as OV
import oracle.sampling as OS
from _helpers import DEV, LSE_ATOL, assert_attn_close, need_gpu
from test_gpu_encode import near_enough, want_of
from test_gpu_kv_weights import i32, tolerance, values
from test_gpu_sampling import tree_of
from tree_verify_attention_gb300 import api

pytestmark = pytest.mark.gpu

N, HQ, HKV, D, V, CAP, KEEP, SINKS, RECENT = 9, 6, 2, 64, 700, 300, 200, 4, 32
ROT, BASE, TEMPERATURE, TOP_K, TOP_P = 32, 1e6, 0.8, 30, 0.95


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


class Loop:
    """Two caches in turn, and what a serving loop keeps beside them."""

    def __init__(self, fmt, start, seed=1):
        g = torch.Generator().manual_seed(seed)
        self.caches = [api.KVCache(HKV, D, CAP, fmt=fmt) for _ in range(2)]
        self.weights = [torch.zeros(HKV, CAP, device=DEV) for _ in range(2)]
        self.caches[0].fill(torch.randn(HKV, start, D, generator=g).to(DEV),
                            torch.randn(HKV, start, D, generator=g).to(DEV))
        self.weights[0][:, :start] = torch.rand(HKV, start, generator=g).to(DEV)
        self.rope = api.Rope(D, ROT, base=BASE)
        self.norms = (1 + 0.2 * torch.randn(2, D, generator=g)).to(DEV)
        self.q, self.k, self.v = (torch.zeros(N, h, D, dtype=torch.bfloat16, device=DEV)
                                  for h in (HQ, HKV, HKV))
        self.step = api.VerifyStep(N, HQ, HKV, D, 0, CAP, V, fmt=fmt,
                                   sampling=api.Sampling(TEMPERATURE, TOP_K, TOP_P))
        self.kept = torch.full((HKV, KEEP), -9, dtype=torch.int32, device=DEV)

    def encode(self, at, x, parent, stream=None):
        c = self.caches[at]
        api.qk_norm_rope(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], self.rope, self.q, self.k,
                         self.v, *self.norms, ctx_len=c.ctx_len, dropped=c.dropped, parent=parent,
                         status=self.step.status, stream=stream)

    def verify(self, at, parent, tokens, x, u, stream=None):
        self.step.run(self.caches[at], self.q, self.k, self.v, parent, tokens, x, uniform=u,
                      stream=stream)

    def weigh(self, at, stream=None):
        s, w = self.step, self.weights[at]
        api.kv_weights(self.caches[at], self.q, s.lse, w, prev=w, decay=0.9, path=s.path,
                       accept_len=s.accept_len, status=s.status, stream=stream)

    def evict(self, at, stream=None):
        api.kv_evict(self.caches[at], self.weights[at], self.caches[1 - at], self.kept,
                     sinks=SINKS, recent=RECENT, weights_out=self.weights[1 - at],
                     status=self.step.status, stream=stream)

    def turn(self, at, inputs, stream=None):
        x, parent, tokens, logits, u = inputs
        self.encode(at, x, parent, stream)
        self.verify(at, parent, tokens, logits, u, stream)
        self.weigh(at, stream)
        self.evict(at, stream)

    def state(self):
        return [t.clone() for t in (
            *(c.k for c in self.caches), *(c.v for c in self.caches),
            *(c.ctx_len for c in self.caches), *(c.dropped for c in self.caches), *self.weights,
            self.q, self.step.out, self.step.argmax, self.step.path, self.kept)]


def inputs(seed):
    """One projection [N, Hq + 2 Hkv, D], a tree whose nodes often carry their
    parents' draws, logits and random numbers."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, HQ + 2 * HKV, D, generator=g).to(torch.bfloat16).to(DEV)
    logits = (3 * torch.randn(N, V, generator=g)).to(torch.bfloat16).to(DEV)
    u = torch.rand(N, generator=g).to(DEV)
    drawn = torch.empty(N, dtype=torch.int32, device=DEV)
    api.sample_tokens(logits, u, api.Sampling(TEMPERATURE, TOP_K, TOP_P), drawn)
    parent, drawn = tree_of(seed, N), drawn.tolist()
    tokens = [0] + [drawn[parent[i]] if i % 3 else 1 for i in range(1, N)]
    return x, i32(parent), i32(tokens), logits, u


@pytest.mark.parametrize("fmt", ["q4_0", "f16"])
def test_every_part_of_a_run(fmt):
    loop = Loop(fmt, 250)
    place, moved = 250, 0       # tokens of the sequence so far; rows that were dropped
    st = loop.step
    for t in range(8):
        at = t % 2
        cache, w = loop.caches[at], loop.weights[at]
        C = int(cache.ctx_len)
        assert int(cache.dropped) == place - C
        ins = inputs(100 + t)
        x, parent, tokens, logits, u = ins
        par = parent.tolist()
        k0, v0 = values(cache, C), values(cache, C, "v")
        old = w.double().cpu().numpy()
        loop.encode(at, x, parent)
        freq = [BASE ** (-2.0 * i / ROT) for i in range(ROT // 2)]
        pos = place + OE.depths(par)
        for src, out, nw in ((x[:, :HQ], loop.q, 0), (x[:, HQ:HQ + HKV], loop.k, 1)):
            near_enough(out, *want_of(src, loop.norms[nw], 1e-6, pos, freq, False),
                        torch.bfloat16)
        assert torch.equal(loop.v, x[:, HQ + HKV:])
        loop.verify(at, parent, tokens, logits, u)
        q, k, v = (a.double().cpu().numpy() for a in (loop.q, loop.k, loop.v))
        out, lse = oracle.attention.tree_verify_attention(q, k0, v0, k, v, par, C, 0)
        assert_attn_close(st.out.cpu().numpy(), out)
        assert np.abs(st.lse.double().cpu().numpy() - lse).max() <= LSE_ATOL
        for i in range(N):
            want, lp, dist = OS.draw(logits[i].float().cpu().numpy(), float(u[i]),
                                     float(np.float32(TEMPERATURE)), TOP_K,
                                     float(np.float32(TOP_P)), 0.0)
            assert dist <= 2.0 ** -29 + V * 2.0 ** -43 or int(st.argmax[i]) == want
        path, emitted = OS.walk(par, tokens.tolist(), st.argmax.tolist())
        a = len(path)
        assert int(st.accept_len) == a and st.path.tolist()[:a] == path
        assert st.out_tokens.tolist()[:a] == emitted
        C, place = C + a, place + a
        assert int(cache.ctx_len) == C
        loop.weigh(at)
        kk = values(cache, C)
        assert np.array_equal(kk[:, :C - a], k0)
        qa, la = q[path], st.lse.double().cpu().numpy()[path]
        decay = float(np.float32(0.9))
        ref = OV.weights(qa, la, kk, old[:, :C], decay)
        had = decay * old[:, :C]
        had[:, C - a:] = 0
        tol = tolerance(qa, la, kk, had, 0, 1 / math.sqrt(D), D, ref)
        got = w.double().cpu().numpy()
        assert np.all(np.abs(got[:, :C] - ref) <= tol)
        loop.evict(at)
        into = loop.caches[1 - at]
        n = min(C, KEEP)
        moved += C > KEEP
        assert int(into.ctx_len) == n and int(into.dropped) == place - n
        wn = w.cpu().numpy()
        for h in range(HKV):
            want = OV.kept(wn[h, :C], KEEP, SINKS, RECENT)
            assert loop.kept[h, :n].tolist() == want
            idx = torch.tensor(want, device=DEV)
            assert torch.equal(into.k[h, :n], cache.k[h, idx])
            assert torch.equal(into.v[h, :n], cache.v[h, idx])
            assert np.array_equal(loop.weights[1 - at][h, :n].cpu().numpy(), wn[h, want])
        assert int(st.status) == 0
    assert moved >= 7


@pytest.mark.parametrize("fmt", ["q4_0", "f16"])
def test_replayed(fmt):
    """Two turns in a graph, there and back, against the same calls one by one."""
    eager, loop = Loop(fmt, 250), Loop(fmt, 250)
    ins = [inputs(7), inputs(8)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for at in (0, 1):
            loop.turn(at, ins[at])
    for _ in range(4):
        g.replay()
        for at in (0, 1):
            eager.turn(at, ins[at])
        for a, b in zip(loop.state(), eager.state()):
            assert torch.equal(a, b)
        # other inputs in the same tensors
        new = [inputs(int(loop.caches[0].dropped)), inputs(1 + int(loop.caches[0].dropped))]
        for old, now in zip(ins, new):
            for a, b in zip(old, now):
                a.copy_(b)
    assert int(loop.step.status) == 0


def test_two_sequences_at_once():
    """Each on its stream, with its own caches, workspaces and outputs."""
    ins = [[inputs(20 + 10 * s + t) for t in range(6)] for s in range(2)]
    want = []
    for s in range(2):
        loop = Loop("q4_0", 250, seed=s)
        for t in range(6):
            loop.turn(t % 2, ins[s][t])
        want.append(loop.state())
    loops = [Loop("q4_0", 250, seed=s) for s in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for t in range(6):
        for s in range(2):
            loops[s].turn(t % 2, ins[s][t], streams[s])
    torch.cuda.synchronize()
    for s in range(2):
        for a, b in zip(loops[s].state(), want[s]):
            assert torch.equal(a, b)
