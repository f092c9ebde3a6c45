"""Attention over the 8-bit cache on the GPU against the float64 definition
(``oracle/attention.py`` over the values of ``oracle/int8.py``).

Tolerances, per output element. With A = sum_j p_j |v_j| of the element:

* weights are rounded to binary16 (2^-11 each, the normaliser is not), and
  2^x, its argument and the scales add 2^-20 together: A (2^-11 + 2^-20);
* a score is a float32 sum of D exact products; each 16-product step may lose
  2^-22 of the largest magnitude it meets, so a score is off by at most
  d = (D / 16 + 4) 2^-22 max_j sum |q k| scale, a weight by 2 d relative:
  2 d A;
* weights under 2^-24 / 2^10 of a slice's largest contribution fall to binary16
  subnormals: 2^-25 of the largest contribution for each of the C keys, below
  2^-12 A for the contexts here;
* a bf16 output rounds to 2^-8 of itself (a float32 one to 2^-24).

The log-sum-exp is off by d + 2^-20 + 2^-22 |lse|.
"""

import numpy as np
import pytest
import torch

import oracle
import oracle.int8 as I8
from _helpers import DEV, need_gpu
from tree_verify_attention_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def rand_tree(rng, n, max_depth=16):
    parent, depth = [-1], [0]
    for i in range(1, n):
        p = int(rng.integers(0, i))
        p = p if depth[p] < max_depth else 0
        parent.append(p)
        depth.append(depth[p] + 1)
    return np.array(parent, np.int32)


class Case:
    """A filled cache and one step's inputs, with the float64 result."""

    def __init__(self, n, hq, hkv, d, ctx, window=0, cap=None, seed=0, parent=None, k_fun=None,
                 v_fun=None, q_scale=1.0, scale=None):
        rng = np.random.default_rng(seed + 1000 * n + ctx)
        self.n, self.hq, self.hkv, self.d, self.ctx, self.window = n, hq, hkv, d, ctx, window
        self.scale = scale

        def bf(x):
            return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)

        k, v = (bf(rng.standard_normal((ctx, hkv, d))) for _ in range(2))
        self.k = k if k_fun is None else k_fun(k.float()).to(torch.bfloat16)
        self.v = v if v_fun is None else v_fun(v.float()).to(torch.bfloat16)
        self.q = bf(rng.standard_normal((n, hq, d)) * q_scale)
        self.tk, self.tv = (bf(rng.standard_normal((n, hkv, d))) for _ in range(2))
        self.parent = rand_tree(rng, n) if parent is None else np.asarray(parent, np.int32)
        self.cache = api.Int8Cache(hkv, d, cap or ctx + n, device=DEV)
        if ctx:
            self.cache.append(self.k.to(DEV), self.v.to(DEV))

    def run(self, dtype=torch.bfloat16, ws=None, status=0):
        out = torch.full((self.n, self.hq, self.d), 5.0, dtype=dtype, device=DEV)
        lse = torch.full((self.n, self.hq), 5.0, device=DEV)
        if ws is None:
            ws = api.workspace(api.int8_attn_workspace_bytes(
                self.n, self.hq, self.hkv, self.d, self.window, self.cache.capacity), device=DEV)
        self.dev = [t.to(DEV) for t in (self.q, self.tk, self.tv, torch.from_numpy(self.parent))]
        api.tree_verify_attn(self.cache, *self.dev, self.window, 64, out, lse, ws,
                             scale=self.scale or 0.0)
        torch.cuda.synchronize()
        assert int(self.cache.status) == status
        return out.double().cpu().numpy(), lse.double().cpu().numpy()

    def values(self):
        return [I8.cached_values(r.float().permute(1, 0, 2).numpy()) for r in (self.k, self.v)]

    def check(self, dtype=torch.bfloat16, rows=None, **kw):
        """Compares the result (of all nodes, or of the nodes ``rows``)."""
        out, lse = self.run(dtype, **kw)
        k, v = self.values()
        q, tk, tv = (t.double().numpy() for t in (self.q, self.tk, self.tv))
        f = oracle.attention.tree_verify_attention_by_head
        args = (self.parent, self.ctx, self.window, self.scale)
        want, wlse = f(q, k, v, tk, tv, *args)
        mag, _ = f(q, k, np.abs(v), tk, np.abs(tv), *args)
        g = self.hq // self.hkv
        qk = 0.0
        for h in range(self.hkv):
            keys = np.abs(np.concatenate([k[h], tk[:, h]]))
            qk = max(qk, (np.abs(q[:, h * g:(h + 1) * g].reshape(-1, self.d)) @ keys.T).max())
        delta = (self.d / 16 + 4) * 2.0 ** -22 * qk * (self.scale or self.d ** -0.5)
        step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
        sel = slice(None) if rows is None else rows
        tol = mag * (2.0 ** -11 + 2.0 ** -20 + 2 * delta + 2.0 ** -12) + step * np.abs(want) + 1e-30
        bad = np.abs(out - want)[sel] / tol[sel]
        assert np.isfinite(out[sel]).all() and bad.max() <= 1.0, f"{bad.max():.3f} of the tolerance"
        dl = np.abs(lse - wlse)[sel] / (delta + 2.0 ** -20 + 2.0 ** -22 * np.abs(wlse[sel]))
        assert dl.max() <= 1.0, f"lse: {dl.max():.3f} of the tolerance"
        return out, lse


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ctx", [0, 1, 63, 64, 65, 127, 128, 129, 191, 700])
def test_context_lengths(d, ctx):
    Case(5, 4, 2, d, ctx).check()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,hq,hkv", [(1, 1, 1), (1, 6, 1), (1, 24, 4), (3, 16, 1), (23, 24, 4),
                                      (65, 8, 8), (65, 12, 2), (40, 2, 1), (13, 30, 5),
                                      (65, 64, 1), (11, 8, 8)])
def test_heads_and_nodes(d, n, hq, hkv):
    Case(n, hq, hkv, d, 333).check()


@pytest.mark.parametrize("window", [1, 2, 3, 17, 64, 65, 200, 500, 5000])
@pytest.mark.parametrize("ctx", [10, 64, 450])
def test_windows(window, ctx):
    Case(23, 12, 2, 128, ctx, window).check()
    Case(1, 4, 2, 64, ctx, window).check()


@pytest.mark.parametrize("parent", ["chain", "star", "binary"])
def test_trees(parent):
    n = 65
    par = {"chain": [-1] + list(range(n - 1)), "star": [-1] + [0] * (n - 1),
           "binary": [-1] + [(i - 1) // 2 for i in range(1, n)]}[parent]
    Case(n, 6, 1, 64, 127, 40, parent=par).check()
    Case(n, 4, 2, 256, 190, 0, parent=par).check()


def test_float_output_and_given_scale():
    Case(9, 8, 2, 128, 300, scale=0.31).check(torch.float32)
    Case(9, 8, 2, 256, 5000, scale=0.02).check(torch.float32)


@pytest.mark.parametrize("d,ctx,window", [(256, 20000, 0), (128, 20011, 0), (64, 30001, 0),
                                          (256, 9000, 2048)])
def test_slices_of_several_chunks(d, ctx, window):
    Case(23, 12, 2, d, ctx, window).check()
    Case(1, 12, 2, d, ctx, window).check()


def test_one_slice_of_many_chunks():
    """So many tiles that every unit walks all chunks."""
    Case(65, 128, 8, 64, 3000).check()


def test_capacity_far_above_the_context():
    """Most slices are planned for rows that are not there yet."""
    Case(23, 12, 2, 128, 200, cap=50000).check()
    Case(1, 12, 2, 256, 1, cap=50000).check()


def test_growing_scores_move_the_reference():
    """Keys aligned with every query, longer and longer: each chunk outgrows
    the last one's maximum by far more than the threshold."""
    n, hq, d = 3, 2, 64

    def ramp(k):
        up = torch.linspace(0.0, 6.0, k.shape[0])[:, None, None]
        return torch.ones_like(k) * up + 0.1 * k

    c = Case(n, hq, 1, d, 2000, k_fun=ramp)
    c.q = (torch.ones(n, hq, d) + 0.1 * c.q.float()).to(torch.bfloat16)
    c.check()
    c = Case(n, hq, 1, d, 2000, k_fun=lambda k: ramp(k).flip(0))
    c.q = (torch.ones(n, hq, d) + 0.1 * c.q.float()).to(torch.bfloat16)
    c.check()


@pytest.mark.parametrize("which", ["k", "v"])
def test_blocks_of_very_different_size(which):
    """Scales from 2^-20 to 2^20, and zero blocks."""
    def vary(x):
        e = torch.tensor([0, 20, -20, -60, 7, -7])
        b = torch.arange(x.shape[0]) // 64
        return x * torch.exp2(e[b % 6].float())[:, None, None] * (0.02 if which == "k" else 1.0)

    # scores stay moderate: large keys meet a small query
    Case(7, 4, 2, 128, 900, q_scale=2.0 ** -17 if which == "k" else 1.0,
         **{which + "_fun": vary}).check()


@pytest.mark.parametrize("q_scale,scale", [(2.0 ** 60, 2.0 ** -64), (2.0 ** -60, 2.0 ** 56)])
def test_query_magnitudes(q_scale, scale):
    Case(5, 4, 2, 64, 200, q_scale=q_scale, scale=scale).check()


def test_stale_rows_and_scales_are_not_read():
    """NaN in every place that is not part of the sequence."""
    c = Case(9, 8, 2, 128, 64 * 5 + 20, cap=64 * 12)
    cache, b = c.cache, 5
    cache.k_scale[:, b:] = float("nan")
    cache.v_scale[:, b:] = float("nan")
    for t in (cache.k_tail, cache.v_tail):
        t[:, b % 2, 20:] = float("nan")
        t[:, (b + 1) % 2] = float("inf")
    cache.k[:, b:] = -128
    cache.v[:, b:] = -128
    c.check()


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 2.0 ** 41])
def test_bad_tree_rows_touch_only_who_sees_them(which, value):
    """Node 2 of head 1 is bad: its descendants have no result in the query
    heads of that head, everyone else is right."""
    parent = [-1, 0, 0, 1, 2, 2, 4, 3, 0]
    sees = [2, 4, 5, 6]
    c = Case(9, 6, 2, 128, 150, parent=parent)
    rows = [i for i in range(9) if i not in sees]
    good = Case(9, 6, 2, 128, 150, parent=parent)
    (c.tk if which == "k" else c.tv)[2, 1, 77] = value
    out, lse = c.run(status=api.DEV_NONFINITE)
    ref, rlse = good.check()
    assert np.isnan(out[sees, 3:]).all() and np.isnan(lse[sees, 3:]).all()
    assert np.array_equal(out[rows], ref[rows]) and np.array_equal(out[:, :3], ref[:, :3])
    assert np.array_equal(lse[rows], rlse[rows])


def test_bad_query_rows_touch_only_themselves():
    c, good = Case(9, 6, 2, 128, 150), Case(9, 6, 2, 128, 150)
    c.q[4, 5, 3] = float("nan")
    c.q[7, 0, 9] = float("inf")
    out, lse = c.run()
    ref, rlse = good.check()
    mask = np.ones((9, 6), bool)
    mask[4, 5] = mask[7, 0] = False
    assert np.isnan(out[4, 5]).all() and not np.isfinite(lse[7, 0])
    assert np.array_equal(out[mask], ref[mask]) and np.array_equal(lse[mask], rlse[mask])


def test_bad_trees_and_lengths_are_reported():
    c = Case(4, 2, 1, 64, 100, parent=[-1, 0, 7, 1])
    c.run(status=api.DEV_BAD_TREE)
    c = Case(5, 2, 1, 64, 100, parent=[-1, 0, 1, 2, 3])
    out = torch.empty(5, 2, 64, device=DEV)
    ws = api.workspace(api.int8_attn_workspace_bytes(5, 2, 1, 64, 0, c.cache.capacity))
    c.run()
    api.tree_verify_attn(c.cache, *c.dev, 0, 3, out, None, ws)
    assert int(c.cache.status) == api.DEV_DEPTH
    c.cache.status.zero_()
    c.cache.ctx_len.fill_(c.cache.capacity + 1)
    api.tree_verify_attn(c.cache, *c.dev, 0, 9, out, None, ws)
    assert int(c.cache.status) == api.DEV_CTX
    c.cache.status.zero_()
    c.cache.ctx_len.fill_(-3)
    api.tree_verify_attn(c.cache, *c.dev, 0, 9, out, None, ws)
    assert int(c.cache.status) == api.DEV_CTX


def test_repeats_are_bit_equal_and_the_workspace_needs_no_clearing():
    c = Case(23, 12, 2, 256, 4000)
    ws = torch.full((api.int8_attn_workspace_bytes(23, 12, 2, 256, 0, c.cache.capacity),), 0xFF,
                    dtype=torch.uint8, device=DEV)      # NaN patterns
    a = c.check(ws=ws)
    b = c.run(ws=ws)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_captured_step_follows_the_committed_length():
    """One graph: attention, then the commit of a chain; replays see what the
    one before committed."""
    n, hq, hkv, d = 4, 4, 2, 128
    c = Case(n, hq, hkv, d, 120, cap=400, parent=[-1, 0, 1, 2])
    ref, _ = c.check()
    out = torch.empty(n, hq, d, device=DEV, dtype=torch.bfloat16)
    lse = torch.empty(n, hq, device=DEV)
    ws = api.workspace(api.int8_attn_workspace_bytes(n, hq, hkv, d, 0, 400), device=DEV)
    length = torch.tensor([3], dtype=torch.int32, device=DEV)
    path = torch.arange(n, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.tree_verify_attn(c.cache, *c.dev, 0, 64, out, lse, ws)
        api.kv_commit(c.cache, length, path, c.dev[1], c.dev[2])
    for step in range(5):
        graph.replay()
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()
        if step == 0:
            assert np.array_equal(got, ref)
        k, v = c.values()
        want, _ = oracle.attention.tree_verify_attention_by_head(
            *(t.double().numpy() for t in (c.q,)), k, v, c.tk.double().numpy(),
            c.tv.double().numpy(), c.parent, c.k.shape[0], 0)
        assert np.abs(got - want).max() < 2e-2
        c.k, c.v = torch.cat([c.k, c.tk[:3]]), torch.cat([c.v, c.tv[:3]])
    assert int(c.cache.ctx_len) == 135


def test_two_streams_at_once():
    a, b = Case(23, 12, 2, 256, 6000), Case(9, 8, 2, 128, 7000)
    ra, rb = a.check(), b.check()
    outs = []
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        for c, st in ((a, s[0]), (b, s[1])):
            with torch.cuda.stream(st):
                out = torch.empty(c.n, c.hq, c.d, dtype=torch.bfloat16, device=DEV)
                ws = api.workspace(api.int8_attn_workspace_bytes(
                    c.n, c.hq, c.hkv, c.d, 0, c.cache.capacity), device=DEV)
                api.tree_verify_attn(c.cache, *c.dev, 0, 64, out, None, ws)
                outs.append((c, out))
    torch.cuda.synchronize()
    for c, out in outs:
        assert np.array_equal(out.double().cpu().numpy(), (ra if c is a else rb)[0])


def test_many_lengths_twice():
    """Every hand-over between the kernel's roles, at many chunk counts: two
    runs of each are equal to the bit, and the float64 result is met."""
    rng = np.random.default_rng(11)
    for _ in range(40):
        n, ctx = int(rng.integers(1, 66)), int(rng.integers(0, 6000))
        c = Case(n, 4, 1, int(rng.choice([64, 128, 256])), ctx, int(rng.choice([0, 0, 300, 4000])),
                 seed=int(rng.integers(1000)))
        a, b = c.check(), c.run()
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_offsets_past_31_bits():
    Case(3, 16, 8, 256, 400, cap=1_200_000).check()


@pytest.mark.slow
@pytest.mark.parametrize("n", [1, 23])
def test_long_context_sampled(n):
    """128K positions; sampled rows against the definition in 64 bits."""
    hq, hkv, d, ctx = 24, 4, 256, 131060
    g = torch.Generator(device=DEV).manual_seed(n)
    k, v = (torch.randn(ctx, hkv, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    cache = api.Int8Cache(hkv, d, ctx + n, device=DEV)
    cache.append(k, v)
    kk, vv = (torch.empty(ctx, hkv, d, device=DEV) for _ in range(2))
    cache.read(0, ctx, kk, vv)
    q = torch.randn(n, hq, d, generator=g, device=DEV).to(torch.bfloat16)
    tk, tv = (torch.randn(n, hkv, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    parent = rand_tree(np.random.default_rng(n), n)
    out, lse = torch.empty(n, hq, d, device=DEV), torch.empty(n, hq, device=DEV)
    ws = api.workspace(api.int8_attn_workspace_bytes(n, hq, hkv, d, 0, cache.capacity), device=DEV)
    api.tree_verify_attn(cache, q, tk, tv, torch.from_numpy(parent).to(DEV), 0, 64, out, lse, ws)
    for node, head in ((0, 0), (n - 1, hq - 1), (n // 2, 7)):
        h = head // (hq // hkv)
        line, x = [], node
        while x >= 0:
            line.append(x)
            x = int(parent[x])
        keys = torch.cat([kk[:, h], tk[line, h].float()]).double()
        vals = torch.cat([vv[:, h], tv[line, h].float()]).double()
        s = keys @ q[node, head].double() / d ** 0.5
        p = torch.softmax(s, 0)
        want, mag = p @ vals, p @ vals.abs()
        assert (out[node, head].double() - want).abs().max() <= (2.0 ** -10 * mag).max()
        assert abs(float(lse[node, head]) - float(torch.logsumexp(s, 0))) < 1e-4
