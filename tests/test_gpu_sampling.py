"""Tokens drawn on the GPU against the float64 definition
(``oracle/sampling.py``).

Tolerances. A weight is off by at most 2^-29 of itself (2^t: the table's 2^-32,
the quartic's and the two floats' 2^-30) and one unit, which is at most 2^-43 of
the largest; a border with the part p of the total below it moves by p (1 - p)
2 2^-29 and V units, less than 2^-29 + V 2^-43. Tokens have to be equal wherever the float64 draw is
further than that from a border; a row that is nearer says nothing. Of rows with
k borders at most 2 k (2^-29 + V 2^-43) are, and with top-p as many more as that
distance is a part of the token at the cut: 2e-8 of 2e-6 for the longest rows
here, 8e-9 of 7e-7 for 20001 tokens and top-p 0.999, about one row in a hundred.
Log probabilities: two conversions, a quotient and a logarithm, 2^-22 absolute
beside 2^-23 of the value."""

import math

import numpy as np
import pytest
import torch

import oracle.sampling as OS
from _helpers import DEV, need_gpu
from tree_verify_attention_gb300 import api

pytestmark = pytest.mark.gpu

@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def make(seed, n, v, dtype, scale=2.0, likely=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, v, generator=g) * scale
    for _ in range(likely):
        at = torch.randint(0, v, (n,), generator=g)
        x[torch.arange(n), at] = 6.0 + 9.0 * torch.rand(n, generator=g)
    u = torch.rand(n, generator=g)
    return x.to(dtype).to(DEV), u.to(DEV)


def run(x, u, s, want_logprob=True):
    n = x.shape[0]
    tok = torch.full((n,), -7, dtype=torch.int32, device=DEV)
    lp = torch.full((n,), 7.0, device=DEV) if want_logprob else None
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    api.sample_tokens(x, u, s, tok, lp, status=st)
    return tok.cpu().numpy(), None if lp is None else lp.cpu().numpy(), int(st)


def f32(x):
    return float(np.float32(x))


def check(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, rows=None, few=0, status=0):
    """Rows `rows` (all) against the oracle; at most `few` may lie on a border."""
    s = api.Sampling(temperature, top_k, top_p, min_p)
    tok, lp, st = run(x, u, s)
    assert st == status
    xs, us = x.float().cpu().numpy(), u.cpu().numpy()
    n = len(us)

    def at(p, i):
        return p[i].item() if isinstance(p, torch.Tensor) else p

    border = 2.0 ** -29 + x.shape[1] * 2.0 ** -43
    near = 0
    for i in range(n) if rows is None else rows:
        want, wlp, dist = OS.draw(xs[i], float(us[i]), f32(at(temperature, i)), at(top_k, i),
                                  f32(at(top_p, i)), f32(at(min_p, i)))
        if dist <= border:
            near += 1
            continue
        assert tok[i] == want, (i, tok[i], want, dist)
        if want < 0:
            assert math.isnan(lp[i])
            continue
        assert abs(lp[i] - wlp) <= 2.0 ** -22 + 2.0 ** -23 * abs(wlp), (i, lp[i], wlp)
    assert near <= few, near
    return tok, lp


FILTERS = [dict(), dict(temperature=0.6), dict(temperature=3.0), dict(top_k=1), dict(top_k=7),
           dict(top_k=50, temperature=0.8), dict(top_p=0.9), dict(top_p=0.3, temperature=1.5),
           dict(top_p=0.999), dict(min_p=0.05), dict(min_p=1.0), dict(top_p=0.0),
           dict(top_k=40, top_p=0.95), dict(top_k=40, top_p=0.95, min_p=0.1, temperature=0.7),
           dict(top_k=2000, top_p=0.8, temperature=2.0), dict(temperature=0.0)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v", [(1, 1), (3, 2), (2, 33), (5, 257), (9, 1024), (4, 8191),
                                 (23, 20001), (80, 5003), (400, 777)])
def test_shapes_and_filters(n, v, dtype):
    for k, f in enumerate(FILTERS):
        x, u = make(n * 1000 + v + k, n, v, dtype, likely=3 if k % 2 else 0)
        check(x, u, few=1, **f)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_long_rows(dtype):
    for n, k in ((1, 24), (2, 0), (23, 24), (80, 8)):
        x, u = make(n + k, n, 151936, dtype, likely=k)
        some = range(0, n, max(1, n // 3))
        for f in (dict(), dict(top_p=0.95), dict(top_k=50, top_p=0.95, temperature=0.8),
                  dict(top_p=0.9, min_p=0.02, temperature=0.7), dict(top_k=5000),
                  dict(top_k=30000, top_p=0.9, temperature=2.0), dict(temperature=0.05)):
            check(x, u, rows=some, few=1, **f)


def test_largest_vocabulary():
    for v in (262144, 1 << 19):
        x, u = make(v, 2, v, torch.float32, likely=10)
        check(x, u, top_p=0.9, few=1)
        check(x, u, few=1)
    x = torch.zeros(1, (1 << 19) + 1, device=DEV)
    with pytest.raises(api.DfvError):
        run(x, torch.zeros(1, device=DEV), api.Sampling())


def test_evenly_spaced_numbers_reach_every_token():
    """4096 random numbers over 64 tokens: each is drawn as often as it is likely."""
    g = torch.Generator().manual_seed(1)
    row = torch.randn(64, generator=g)
    x = row.expand(4096, 64).contiguous().to(DEV)
    u = ((torch.arange(4096) + 0.5) / 4096).to(DEV)
    for f in (dict(), dict(top_k=20), dict(top_p=0.7), dict(min_p=0.2)):
        tok, _ = check(x, u, few=0, **f)
        ids, w, _ = OS.kept(row.numpy(), 1.0, f.get("top_k", 0), f32(f.get("top_p", 1.0)),
                            f32(f.get("min_p", 0.0)))
        got = np.bincount(tok, minlength=64)
        assert np.all(np.diff(tok) >= 0) and np.abs(got[ids] - 4096 * w / w.sum()).max() <= 1


def test_ties():
    """Equal logits: the lowest indices are kept, also where thousands are equal."""
    for v in (10, 700, 40000):
        x = torch.zeros(3, v, device=DEV)
        x[:, v // 2] = 1.0
        u = torch.tensor([0.0, 0.5, 0.999], device=DEV)
        for k in (1, 2, 5, v // 3 + 2, v - 1):
            # (k = 39999: the total is 39998 + e, and 0.99900001 of it is 39960.7181, one
            # border 39959 - 1 + e = 39960.7183, nearer than 6.4e-9 of the total)
            check(x, u, top_k=k, few=1 if k == 39999 else 0)
        check(x, u, top_p=0.5)
        check(x, u)
        check(x, u, temperature=0.0)
        # (of an even number of equal tokens, 100 and 5714, half is a border)
        check(torch.full((3, v), -2.0, device=DEV), u, top_k=max(1, v // 7), few=1)
    # -0 equals +0
    x = torch.tensor([[-0.0, 0.0, -0.0, 0.0]], device=DEV)
    tok, _ = check(x, torch.tensor([0.9], device=DEV), top_k=2)
    assert tok[0] == 1
    # values that differ in their last bits: cuts inside a bin of many keys
    g = torch.Generator().manual_seed(3)
    x = (1.0 + 1e-4 * torch.rand(4, 30000, generator=g)).to(DEV)
    u = torch.rand(4, generator=g).to(DEV)
    for f in (dict(top_k=9999), dict(top_p=0.37), dict(top_k=20000, top_p=0.5)):
        check(x, u, few=1, **f)
    # around zero, where keys are far apart
    x = (1e-30 * torch.randn(2, 5000, generator=g)).to(DEV)
    check(x, u[:2], top_k=1234)


def test_masked_logits():
    """-inf and the types' lowest values are never drawn beside others."""
    for dtype in (torch.float32, torch.bfloat16):
        for low in (-math.inf, torch.finfo(dtype).min, -1e4):
            x, u = make(11, 6, 3001, dtype)
            x[:, ::2] = low
            x[4, :] = low
            x[4, 2999] = 0.5
            x[5, :3000] = low
            # (row 5 is masked throughout: no token, or any where the mask is a number)
            st = api.DEV_NONFINITE if low == -math.inf else 0
            for f in (dict(), dict(top_k=2000), dict(top_p=0.9), dict(top_k=3000, top_p=0.99)):
                tok, lp = check(x, u, few=1, status=st, **f)
                assert tok[4] == 2999 and lp[4] == 0.0 and (tok[5] == -1) == bool(st)
    # a row of lowest values alone is uniform
    x = torch.full((2, 1000), torch.finfo(torch.float32).min, device=DEV)
    check(x, torch.tensor([0.2503, 0.5003], device=DEV), top_k=500)


def test_magnitudes():
    """Logits far from zero and temperatures far from one."""
    g = torch.Generator().manual_seed(8)
    z = torch.randn(3, 2000, generator=g)
    u = torch.rand(3, generator=g).to(DEV)
    for add, temp in ((0.0, 1e-3), (1e5, 0.5), (-1e5, 1.0), (1e6, 1.0), (3e4, 0.01), (0.0, 1e4),
                      (0.0, 3e38), (1e30, 1e29)):
        x = (z * (1e29 if add == 1e30 else 1.0) + add).to(DEV)
        for f in (dict(), dict(top_k=100), dict(top_p=0.8)):
            check(x, u, temperature=temp, few=1, **f)
    x = torch.tensor([[3.0, 3.0 + 2.0 ** -20, 1.0]], device=DEV)
    check(x, u[:1], temperature=1e-7)
    check(x, u[:1], temperature=1e-35)       # below 2^-100: greedy


def test_each_row_its_own_parameters():
    n, v = 120, 4000
    x, u = make(21, n, v, torch.bfloat16, likely=4)
    g = torch.Generator().manual_seed(2)

    def pick(values, dt):
        i = torch.randint(0, len(values), (n,), generator=g)
        return torch.tensor(values, dtype=dt)[i].to(DEV)

    t = pick([0.0, 0.5, 1.0, 1.7], torch.float32)
    k = pick([-3, 0, 1, 40, 1000, 4000, 1 << 30], torch.int32)
    p = pick([1.0, 0.9, 0.5, 0.0, -1.0, 2.0], torch.float32)
    m = pick([0.0, 0.02, 0.5, 1.0, 3.0, -1.0], torch.float32)
    check(x, u, t, k, p, m, few=1)
    check(x, u, t, 30, p, 0.01, few=1)


def test_bad_rows_and_parameters():
    x, u = make(5, 12, 500, torch.float32)
    x[1, 7] = math.nan
    x[2, 499] = math.inf
    x[3] = -math.inf
    s = api.Sampling(top_k=20, top_p=0.9)
    tok, lp, st = run(x, u, s)
    clean = [0] + list(range(4, 12))
    assert st == api.DEV_NONFINITE
    assert np.all(tok[1:4] == -1) and np.all(np.isnan(lp[1:4]))
    want = run(x[clean].contiguous(), u[clean].contiguous(), s)
    assert want[2] == 0 and np.array_equal(tok[clean], want[0]) and np.array_equal(lp[clean],
                                                                                  want[1])
    x, u = make(6, 12, 500, torch.float32)
    t = torch.ones(12, device=DEV)
    p, m = torch.ones(12, device=DEV), torch.zeros(12, device=DEV)
    t[0], t[1], t[2] = -1.0, math.nan, math.inf
    p[3], m[4], u[5], u[6], u[7] = math.nan, math.nan, 1.0, -1e-9, math.nan
    tok, lp, st = run(x, u, api.Sampling(t, 0, p, m))
    assert st == api.DEV_BAD_SAMPLING
    assert np.all(tok[:8] == -1) and np.all(np.isnan(lp[:8])) and np.all(tok[8:] >= 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_alignment(dtype):
    for v in (1000, 1001, 5, 4099):
        for off in range(4):
            wide = make(v + off, 6, v + 13, dtype)[0]
            x = wide[:, off:off + v]
            u = torch.rand(6, generator=torch.Generator().manual_seed(off)).to(DEV)
            for f in (dict(), dict(top_k=3), dict(top_p=0.9)):
                check(x, u, few=1, **f)


def test_equal_runs_and_streams():
    x, u = make(31, 23, 50021, torch.bfloat16, likely=2)
    s = api.Sampling(temperature=1.2, top_k=900, top_p=0.97, min_p=1e-4)
    a = run(x, u, s)
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for k in range(4):
        t, lp = torch.empty(23, dtype=torch.int32, device=DEV), torch.empty(23, device=DEV)
        api.sample_tokens(x, u, s, t, lp, stream=side[k % 2])
        outs.append((t, lp))
    torch.cuda.synchronize()
    for t, lp in outs:
        assert np.array_equal(t.cpu().numpy(), a[0]) and np.array_equal(lp.cpu().numpy(), a[1])
    # one row alone is drawn as among others, whatever the split
    for i in (0, 11, 22):
        one = run(x[i:i + 1], u[i:i + 1], s)
        assert one[0][0] == a[0][i] and one[1][0] == a[1][i]
    many = run(x.repeat(20, 1), u.repeat(20), s)
    assert np.array_equal(many[0], np.tile(a[0], 20))
    assert np.array_equal(many[1], np.tile(a[1], 20))


def tree_of(seed, n):
    r = np.random.default_rng(seed)
    return [-1] + [int(r.integers(0, i)) for i in range(1, n)]


@pytest.mark.parametrize("n", [1, 2, 23, 40, 65])
def test_accept(n):
    v = 3000
    for seed, f in enumerate((dict(temperature=0.5, top_k=2), dict(top_p=0.4), dict(),
                              dict(temperature=0.0))):
        x, u = make(seed, n, v, torch.bfloat16, likely=1)
        parent = tree_of(seed, n)
        target, lp, _ = run(x, u, api.Sampling(**f))
        r = np.random.default_rng(seed + 5)
        tokens = [0] + [int(target[parent[i]]) if r.random() < 0.7 else 1 for i in range(1, n)]
        ws = api.workspace(api.sample_accept_workspace_bytes(n, v), device=DEV)
        ti = torch.tensor(tokens, dtype=torch.int32, device=DEV)
        pi = torch.tensor(parent, dtype=torch.int32, device=DEV)
        for _ in range(3):     # the workspace is ready again after each call
            out = [torch.full((n,), -9, dtype=torch.int32, device=DEV) for _ in range(3)]
            ln = torch.zeros(1, dtype=torch.int32, device=DEV)
            l2 = torch.empty(n, device=DEV)
            api.sample_accept(x, u, api.Sampling(**f), pi, ti, out[0], ln, out[1], out[2], ws,
                              logprob=l2)
            path, emitted = OS.walk(parent, tokens, target)
            assert np.array_equal(out[0].cpu().numpy(), target)
            assert np.array_equal(l2.cpu().numpy(), lp)
            assert int(ln) == len(path)
            assert out[1].tolist() == path + [-1] * (n - len(path))
            assert out[2].tolist() == emitted + [-1] * (n - len(path))
        assert not ws.any()


def test_accept_with_bad_rows_and_parents():
    n, v = 5, 100
    x, u = make(3, n, v, torch.float32)
    x[0] = -math.inf                    # no token at the root: nothing follows it
    s = api.Sampling()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = [torch.full((n,), -9, dtype=torch.int32, device=DEV) for _ in range(3)]
    ln = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = api.workspace(256, device=DEV)
    minus = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    parent = torch.tensor([9, 7, -4, 0, 3], dtype=torch.int32, device=DEV)
    api.sample_accept(x, u, s, parent, minus, out[0], ln, out[1], out[2], ws, status=st)
    assert int(st) == api.DEV_NONFINITE | api.DEV_BAD_TREE
    assert int(ln) == 1 and out[1].tolist() == [0, -1, -1, -1, -1] and out[2].tolist() == [-1] * 5


def test_graph():
    n, v = 23, 20000
    x, u = make(9, n, v, torch.bfloat16, likely=3)
    t = torch.ones(n, device=DEV)
    s = api.Sampling(temperature=t, top_p=0.9)
    parent = torch.tensor(tree_of(1, n), dtype=torch.int32, device=DEV)
    tokens = torch.zeros(n, dtype=torch.int32, device=DEV)
    out = [torch.full((n,), -9, dtype=torch.int32, device=DEV) for _ in range(3)]
    ln = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = api.workspace(256, device=DEV)
    api.sample_accept(x, u, s, parent, tokens, out[0], ln, out[1], out[2], ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.sample_accept(x, u, s, parent, tokens, out[0], ln, out[1], out[2], ws)
    for k in range(3):                  # new numbers and temperatures, the same graph
        u.copy_(make(40 + k, n, 2, torch.float32)[1])
        t.fill_(0.5 + 0.4 * k)
        g.replay()
        want, _, _ = run(x, u, s)
        assert np.array_equal(out[0].cpu().numpy(), want)
        path, _ = OS.walk(parent.tolist(), tokens.tolist(), want)
        assert int(ln) == len(path)


@pytest.mark.parametrize("fmt", ["q4_0", "f16", "int8"])
def test_sampled_steps(fmt):
    """Chained steps that draw: attention as the greedy step's, the walk along
    the drawn tokens, the accepted rows in the cache."""
    n, hq, hkv, d, v, cap = 9, 4, 2, 64, 500, 400
    g = torch.Generator().manual_seed(7)

    def rows(*shape):
        return torch.randn(*shape, generator=g).to(torch.bfloat16).to(DEV)

    caches = [api.Int8Cache(hkv, d, cap) if fmt == "int8" else api.KVCache(hkv, d, cap, fmt=fmt)
              for _ in range(2)]
    k0, v0 = rows(hkv, 200, d), rows(hkv, 200, d)
    for c in caches:
        c.fill(k0, v0)
    s = api.Sampling(temperature=0.8, top_k=20)
    step = api.VerifyStep(n, hq, hkv, d, 0, cap, v, fmt=fmt, sampling=s, top=3)
    plain = api.VerifyStep(n, hq, hkv, d, 0, cap, v, fmt=fmt)
    length = 200
    for k in range(4):
        q, tk, tv = rows(n, hq, d), rows(n, hkv, d), rows(n, hkv, d)
        x, u = make(60 + k, n, v, torch.bfloat16, likely=1)
        parent = tree_of(k, n)
        target, lp, _ = run(x, u, s)
        tokens = [0] + [int(target[parent[i]]) for i in range(1, n)]
        pi = torch.tensor(parent, dtype=torch.int32, device=DEV)
        ti = torch.tensor(tokens, dtype=torch.int32, device=DEV)
        step.run(caches[0], q, tk, tv, pi, ti, x, uniform=u)
        path, emitted = OS.walk(parent, tokens, target)
        assert int(step.status) == 0
        assert step.path.tolist()[:len(path)] == path and int(step.accept_len) == len(path)
        assert step.out_tokens.tolist()[:len(path)] == emitted
        assert np.array_equal(step.argmax.cpu().numpy(), target)
        assert np.array_equal(step.draw_logprob.cpu().numpy(), lp)
        # a greedy step over logits that make the drawn tokens the largest
        y = torch.zeros(n, v, device=DEV)
        y[torch.arange(n), torch.from_numpy(target).long().to(DEV)] = 1.0
        plain.run(caches[1], q, tk, tv, pi, ti, y)
        length += len(path)
        assert torch.equal(step.out, plain.out) and torch.equal(step.path, plain.path)
        assert int(caches[0].ctx_len) == int(caches[1].ctx_len) == length
        if fmt != "int8":
            assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)


def test_refusals():
    x, u = make(1, 4, 100, torch.float32)
    t = torch.full((4,), -7, dtype=torch.int32, device=DEV)
    s = api.Sampling()

    def no(*a, **kw):
        with pytest.raises(api.DfvError):
            api.sample_tokens(*a, **kw)

    no(x.half(), u, s, t)
    no(x[0], u, s, t)
    no(x.t(), u, s, t)
    no(x.cpu(), u, s, t)
    no(x, u[:3], s, t)
    no(x, u.double(), s, t)
    no(x, u, s, t.long())
    no(x, u, s, t[:3])
    no(x, u, None, t)
    no(x, u, dict(temperature=1.0), t)
    no(x, u, s, t, torch.empty(3, device=DEV))
    no(x, u, api.Sampling(temperature=torch.ones(3, device=DEV)), t)
    for kw in (dict(temperature=-0.1), dict(temperature=math.nan), dict(temperature=math.inf),
               dict(top_p=math.nan), dict(min_p=math.nan), dict(temperature=torch.ones(4)),
               dict(top_k=torch.ones(4, device=DEV)), dict(top_p=u.double())):
        with pytest.raises(api.DfvError):
            api.Sampling(**kw)
    ws = api.workspace(256, device=DEV)
    i = [torch.zeros(4, dtype=torch.int32, device=DEV) for _ in range(5)]
    for bad in (dict(ws=ws[:100]), dict(ws=ws[16:]), dict(parent=i[0][:3]), dict(path=i[3].long())):
        a = dict(parent=i[0], tokens=i[1], accept_len=i[2], path=i[3], out_tokens=i[4], ws=ws)
        a.update(bad)
        with pytest.raises(api.DfvError):
            api.sample_accept(x, u, s, a["parent"], a["tokens"], t, a["accept_len"], a["path"],
                              a["out_tokens"], a["ws"])
    with pytest.raises(api.DfvError):
        api.VerifyStep(4, 4, 2, 64, 0, 100, 100, sampling=s, pipelined=True)
    with pytest.raises(api.DfvError):
        api.VerifyStep(4, 4, 2, 64, 0, 100, 100, sampling=1.0)
    assert torch.all(t == -7)
    api.sample_tokens(x[:0], u[:0], s, t[:0])


def test_steps_over_bit_patterns():
    """bf16 logits given as int16, as the greedy step takes them; and rows that
    have no distribution, whose scores are NaN."""
    n, hq, hkv, d, v, cap = 5, 4, 2, 64, 600, 50
    q, tk = torch.zeros(n, hq, d, dtype=torch.bfloat16, device=DEV), torch.zeros(
        n, hkv, d, dtype=torch.bfloat16, device=DEV)
    x, u = make(3, n, v, torch.bfloat16)
    x[2, 5] = math.nan
    parent = torch.tensor([-1, 0, 1, 2, 3], dtype=torch.int32, device=DEV)
    tokens = torch.zeros(n, dtype=torch.int32, device=DEV)
    got = []
    for y in (x, x.view(torch.int16)):
        step = api.VerifyStep(n, hq, hkv, d, 0, cap, v, sampling=api.Sampling(top_p=0.9), top=2)
        step.run(api.KVCache(hkv, d, cap), q, tk, tk, parent, tokens, y, uniform=u)
        got.append([step.argmax, step.path, step.accept_len, step.status])
        assert int(step.argmax[2]) == -1 and torch.isnan(step.draw_logprob[2])
        assert int(step.status) & api.DEV_NONFINITE
        good = torch.tensor([0, 1, 3, 4], device=DEV)
        assert torch.all(step.argmax[good] >= 0) and torch.all(torch.isfinite(step.logprob[good]))
        assert torch.isnan(step.logprob[2])
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("t", [1e-30, 1e-6, 1e6, 3e38])
def test_extreme_temperatures(t):
    """All the mass on the maximum, or on all alike."""
    x, u = make(9, 6, 5000, torch.float32)
    tok, _ = check(x, u, temperature=t, few=0)
    check(x * 1e30, u, temperature=t, few=0)
    if t < 1:
        assert np.array_equal(tok, x.argmax(1).cpu().numpy())
