"""The 8-bit operators on two streams that fork and join, eagerly and captured
into one graph: what joins waits for both, although every kernel may be set up
early."""

import pytest
import torch

from _helpers import DEV, need_gpu
from tree_verify_attention_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


class Work:
    """Two caches written on two streams, an attention over each behind the
    other's stream, and log probabilities of a row that both precede."""

    def __init__(self):
        g = torch.Generator(device=DEV).manual_seed(7)
        self.rows = torch.randn(3000, 4, 128, generator=g, device=DEV).to(torch.bfloat16)
        self.q = torch.randn(5, 8, 128, generator=g, device=DEV).to(torch.bfloat16)
        self.parent = torch.tensor([-1, 0, 1, 0, 3], dtype=torch.int32, device=DEV)
        self.caches = [api.Int8Cache(4, 128, 4000, device=DEV) for _ in range(2)]
        self.out = [torch.empty(5, 8, 128, device=DEV) for _ in range(2)]
        self.lse = [torch.empty(5, 8, device=DEV) for _ in range(2)]
        self.ws = [api.workspace(api.int8_attn_workspace_bytes(5, 8, 4, 128, 0, 4000))
                   for _ in range(2)]
        self.logits = torch.randn(40, 30000, generator=g, device=DEV)
        self.lp = torch.empty(40, device=DEV)
        self.ids = torch.empty(40, 5, dtype=torch.int32, device=DEV)
        self.tokens = torch.arange(40, dtype=torch.int32, device=DEV)
        self.back = [torch.empty(100, 4, 128, device=DEV) for _ in range(2)]

    def run(self, side):
        main = torch.cuda.current_stream()
        a, b = self.caches
        tree = self.rows[:5]
        fork, there, here = (torch.cuda.Event() for _ in range(3))
        fork.record(main)
        side.wait_event(fork)
        a.append(self.rows, self.rows, at=0)
        b.append(self.rows[:2000], self.rows[:2000], at=0, stream=side)
        api.token_logprobs(self.logits, self.tokens, self.lp, None, self.ids, stream=side)
        there.record(side)
        here.record(main)
        main.wait_event(there)
        side.wait_event(here)
        api.tree_verify_attn(b, self.q, tree, tree, self.parent, 0, 5, self.out[1], self.lse[1],
                             self.ws[1])
        api.tree_verify_attn(a, self.q, tree, tree, self.parent, 0, 5, self.out[0], self.lse[0],
                             self.ws[0], stream=side)
        a.read(2900, 100, *self.back, stream=side)
        joined = torch.cuda.Event()
        joined.record(side)
        main.wait_event(joined)

    def results(self):
        return [t.clone() for t in (*self.out, *self.lse, *self.back, self.lp, self.ids)]

    def wipe(self):
        for t in (*self.out, *self.lse, *self.back, self.lp, self.ids):
            t.zero_()
        for c in self.caches:
            c.k.zero_(), c.v.zero_(), c.open_end.zero_()


def test_two_streams_forked_and_joined():
    w, side = Work(), torch.cuda.Stream()
    # one call after the other, for comparison
    w.caches[0].append(w.rows, w.rows, at=0)
    w.caches[1].append(w.rows[:2000], w.rows[:2000], at=0)
    tree = w.rows[:5]
    for c, o, l, ws in zip(w.caches, w.out, w.lse, w.ws):
        torch.cuda.synchronize()
        api.tree_verify_attn(c, w.q, tree, tree, w.parent, 0, 5, o, l, ws)
    api.token_logprobs(w.logits, w.tokens, w.lp, None, w.ids)
    w.caches[0].read(2900, 100, *w.back)
    torch.cuda.synchronize()
    want = w.results()
    for _ in range(5):
        w.wipe()
        w.run(side)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, w.results()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.run(side)
    for _ in range(5):
        w.wipe()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, w.results()))
    assert all(int(c.status) == 0 for c in w.caches)
