"""Weights that cached keys receive, on the GPU against the float64 definition
(``oracle/eviction.py``).

Tolerance of a term exp(x - lse), x = scale q . k: products are exact (K in two
parts) and added in float32 over D / 16 steps for each part, each within 2^-23
of the running magnitude, so x is off by at most D / 8 * 2^-23 scale sum |q k|;
slope, offset and their sum add 2^-23 (|x| + |lse|) each at most, ex2.approx 2^-22
and the sum of n group terms n group 2^-24 of the total."""

import math

import numpy as np
import pytest
import torch

import oracle
import oracle.eviction as OV
from _helpers import DEV, need_gpu
from tree_verify_attention_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make(seed, hkv, d, C, cap, fmt, n, hq, scale=1.0):
    """A cache of C rows, its K values, queries and their lse over all C keys."""
    g = torch.Generator().manual_seed(seed)
    cache = api.KVCache(hkv, d, cap, fmt=fmt)
    if C:
        cache.fill(torch.randn(hkv, C, d, generator=g).to(DEV),
                   torch.randn(hkv, C, d, generator=g).to(DEV))
    k = values(cache, C)
    q = (torch.randn(n, hq, d, generator=g) * scale).to(torch.bfloat16)
    qd = q.double().numpy()
    lse = np.zeros((n, hq))
    for h in range(hq):
        x = qd[:, h] @ k[h // (hq // hkv)].T / math.sqrt(d) if C else np.zeros((n, 1))
        lse[:, h] = np.log(np.exp(x - x.max(1, keepdims=True)).sum(1)) + x.max(1)
    lse = torch.from_numpy(lse).float().to(DEV)
    prev = torch.rand(hkv, cap, generator=g).to(DEV)
    return cache, k, q.to(DEV), lse, prev


def values(cache, C, which="k"):
    b = getattr(cache, which)[:, :C].cpu().numpy()
    if cache.fmt == "f16":
        return b.view(np.float16).astype(np.float64)
    h, d = cache.n_kv_heads, cache.head_dim
    return oracle.q4_0.dequantize_rows(b.reshape(h, C, d // 32, 18)).astype(np.float64)


def tolerance(q, lse, k, had, window, scale, d, ref):
    n, hq, _ = q.shape
    hkv, C, _ = k.shape
    tol = 2.0 ** -22 * np.abs(had) + (n * hq // hkv + 8) * 2.0 ** -24 * np.abs(ref)
    for s in range(n):
        at = C - n + s
        lo = 0 if window == 0 else max(0, at - window + 1)
        for h in range(hq):
            if at < 0 or not (np.isfinite(lse[s, h]) and np.isfinite(q[s, h]).all()):
                continue
            g = h // (hq // hkv)
            x = scale * (k[g, lo:at + 1] @ q[s, h])
            a = scale * (np.abs(k[g, lo:at + 1]) @ np.abs(q[s, h]))
            e = d / 8 * 2.0 ** -23 * a + 2.0 ** -22 * (np.abs(x) + abs(lse[s, h])) + 2.0 ** -21
            tol[g, lo:at + 1] += np.exp(x - lse[s, h]) * e
    return tol


def check(seed, hkv, hq, d, C, fmt, n, cap=None, decay=1.0, window=0, with_prev=True,
          in_place=False, rows=None):
    cap = cap or C + 7
    cache, k, q, lse, prev = make(seed, hkv, d, C, cap, fmt, n, hq)
    out = prev if in_place else torch.full((hkv, cap), -5.0, device=DEV)
    old = prev.double().cpu().numpy()
    st = i32([0])
    api.kv_weights(cache, q, lse, out, prev=prev if with_prev else None, decay=decay,
                   window=window, status=st)
    qn, ln = q.double().cpu().numpy(), lse.double().cpu().numpy()
    ref = OV.weights(qn, ln, k, old[:, :C] if with_prev else None, decay, window)
    had = decay * old[:, :C] if with_prev else np.zeros((hkv, C))
    tol = tolerance(qn, ln, k, had, window, 1 / math.sqrt(d), d, ref)
    got = out.double().cpu().numpy()
    assert int(st) == 0
    assert np.all(np.abs(got[:, :C] - ref) <= tol), np.max(np.abs(got[:, :C] - ref) / (tol + 1e-30))
    assert np.array_equal(got[:, C:], old[:, C:] if in_place else np.full((hkv, cap - C), -5.0))


@pytest.mark.parametrize("fmt", ["q4_0", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_shapes(fmt, d):
    for k, (hkv, hq, C, n) in enumerate(((1, 1, 1, 1), (2, 12, 100, 1), (4, 24, 1000, 9),
                                         (3, 3, 129, 5), (8, 32, 257, 17), (1, 8, 640, 65),
                                         (2, 10, 128, 3), (5, 5, 3001, 2))):
        check(k, hkv, hq, d, C, fmt, n)


@pytest.mark.parametrize("fmt", ["q4_0", "f16"])
def test_capacities_of_any_alignment(fmt):
    """Heads whose rows start on 4- and 8-byte boundaries, chunks that end anywhere."""
    for d in (64, 128):
        for C in (5, 127, 130, 255, 383):
            for cap in (C, C + 1, C + 2, C + 3):
                check(C + cap, 3, 6, d, C, fmt, 2, cap=cap)


@pytest.mark.parametrize("fmt,d,hkv,hq,n", [("q4_0", 256, 4, 24, 65), ("f16", 128, 8, 32, 65),
                                            ("q4_0", 64, 2, 16, 200), ("f16", 256, 1, 8, 33)])
def test_more_query_rows_than_a_tile(fmt, d, hkv, hq, n):
    check(n, hkv, hq, d, 700, fmt, n, decay=0.75)


@pytest.mark.parametrize("fmt", ["q4_0", "f16"])
def test_many_chunks(fmt):
    """Several chunks, heads and tiles to a CTA."""
    check(1, 8, 8, 64, 30011, fmt, 2, decay=0.9)
    check(2, 8, 16, 64, 9001, fmt, 70)


@pytest.mark.parametrize("fmt", ["q4_0", "f16"])
def test_windows(fmt):
    for C, n, w in ((1000, 5, 1), (1000, 5, 3), (1000, 9, 64), (1000, 2, 257), (1000, 1, 5000),
                    (300, 65, 17), (40, 3, 40), (5000, 4, 1300)):
        check(C + w, 2, 6, 128, C, fmt, n, window=w, decay=0.5)


def test_prev_decay_and_in_place():
    for fmt in ("q4_0", "f16"):
        check(3, 2, 4, 256, 400, fmt, 3, with_prev=False)
        check(4, 2, 4, 256, 400, fmt, 3, decay=0.0)
        check(5, 2, 4, 256, 400, fmt, 3, decay=1.25, in_place=True)
        check(6, 2, 16, 256, 400, fmt, 40, in_place=True)          # several tiles


def test_more_rows_than_keys():
    for C, n in ((1, 3), (2, 9), (5, 5), (130, 200)):
        check(C, 2, 4, 64, C, "q4_0", n)


def test_no_keys():
    for window in (0, 5):
        cache, _, q, lse, prev = make(1, 2, 64, 0, 50, "f16", 3, 4)
        out = torch.full((2, 50), -5.0, device=DEV)
        api.kv_weights(cache, q, lse, out, prev=prev, window=window)
        assert torch.all(out == -5.0)


def test_accepted_nodes():
    """path and accept_len pick the rows; a bad entry counts for nothing."""
    hkv, hq, d, C, n = 2, 12, 256, 500, 23
    cache, k, q, lse, prev = make(9, hkv, d, C, C, "q4_0", n, hq)
    path = [0, 3, 7, 8, 20] + [-1] * 18
    for L in (1, 3, 5):
        out, st = torch.empty(hkv, C, device=DEV), i32([0])
        api.kv_weights(cache, q, lse, out, prev=prev, path=i32(path), accept_len=i32([L]),
                       status=st)
        want = torch.empty(hkv, C, device=DEV)
        at = path[:L]
        api.kv_weights(cache, q[at].contiguous(), lse[at].contiguous(), want, prev=prev)
        assert int(st) == 0
        if L * hq // hkv > 16:
            assert torch.equal(out, want)
        else:   # up to 16 rows of a head are summed in another order: each within its tolerance
            qn, ln = (t[at].double().cpu().numpy() for t in (q, lse))
            ref = OV.weights(qn, ln, k, prev.double().cpu().numpy())
            had = prev.double().cpu().numpy()
            tol = tolerance(qn, ln, k, had, 0, 1 / math.sqrt(d), d, ref)
            for x in (out, want):
                assert np.all(np.abs(x.double().cpu().numpy() - ref) <= tol)
    for L, now in ((0, 0), (24, 23), (-1, 0)):
        out, st = torch.empty(hkv, C, device=DEV), i32([0])
        api.kv_weights(cache, q, lse, out, prev=prev, accept_len=i32([L]), status=st)
        want = prev.clone()
        if now:
            api.kv_weights(cache, q, lse, want, prev=prev)
        assert torch.equal(out, want)
        assert int(st) == (0 if L == 0 else api.DEV_BAD_PATH)
    out, st = torch.empty(hkv, C, device=DEV), i32([0])
    api.kv_weights(cache, q, lse, out, path=i32([0, 23, 7, -5] + [0] * 19), accept_len=i32([4]),
                   status=st)
    l2 = lse[[0, 1, 7, 1]].clone()
    l2[1] = l2[3] = math.inf
    want = torch.empty(hkv, C, device=DEV)
    api.kv_weights(cache, q[[0, 1, 7, 1]].contiguous(), l2, want)
    assert int(st) == api.DEV_BAD_PATH and torch.equal(out, want)


def test_rows_that_are_not_finite():
    hkv, hq, d, C, n = 2, 6, 128, 300, 4
    for fmt in ("q4_0", "f16"):
        cache, k, q, lse, _ = make(2, hkv, d, C, C, fmt, n, hq)
        q[1, 2, 5] = math.inf
        q[2, 0, 0] = math.nan
        lse[3, 5], lse[0, 4], lse[0, 1] = math.nan, math.inf, -math.inf
        out, st = torch.empty(hkv, C, device=DEV), i32([0])
        api.kv_weights(cache, q, lse, out, status=st)
        assert int(st) == api.DEV_NONFINITE
        qn, ln = q.double().cpu().numpy(), lse.double().cpu().numpy()
        ref = OV.weights(qn, ln, k, None)
        tol = tolerance(qn, ln, k, 0 * ref, 0, 1 / math.sqrt(d), d, ref)
        assert np.all(np.abs(out.double().cpu().numpy() - ref) <= tol)


def test_magnitudes_of_queries():
    """Queries of any size: a power of two moved into the scale changes nothing."""
    hkv, hq, d, C, n = 1, 4, 64, 200, 3
    cache, k, q, lse, _ = make(5, hkv, d, C, C, "q4_0", n, hq)
    want = torch.empty(hkv, C, device=DEV)
    api.kv_weights(cache, q, lse, want, scale=0.125)
    for e in (-60, -20, 20, 60, 100):
        out = torch.empty(hkv, C, device=DEV)
        api.kv_weights(cache, q * 2.0 ** e, lse, out, scale=0.125 * 2.0 ** -e)
        assert torch.equal(out, want)
    # and each row has its own
    f = (2.0 ** torch.tensor([-30.0, 0.0, 30.0]))[:, None, None].to(DEV)
    parts = torch.zeros(hkv, C, dtype=torch.float64, device=DEV)
    out = torch.empty(hkv, C, device=DEV)
    for s in range(n):
        l2 = lse.clone()
        l2[:s], l2[s + 1:] = math.inf, math.inf
        api.kv_weights(cache, (q * f).to(torch.bfloat16), l2, out, scale=0.125 * 2.0 ** (30 - 30 * s))
        parts += out.double()
    assert torch.allclose(parts.float(), want, rtol=1e-6)


def test_a_step_and_the_weights_of_its_rows():
    """After a verify step: its lse, path and accept_len give weights that sum to
    one for each accepted node and query head (a chain: all that a node sees is
    cached). The cached rows differ from the attended bf16 ones by a rounding to
    binary16 below 2^-11 of a value: a score by 2^-11 scale sum |q k|."""
    n, hq, hkv, d, C = 6, 8, 2, 128, 777
    cache, k, _, _, _ = make(7, hkv, d, C, C + n, "f16", 1, hq)
    g = torch.Generator().manual_seed(3)

    def rows(*s):
        return torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)

    q, tk, tv = rows(n, hq, d), rows(n, hkv, d), rows(n, hkv, d)
    parent = i32([-1, 0, 1, 2, 3, 4])
    v = 64
    logits = torch.zeros(n, v, device=DEV)
    tokens = i32([0, 1, 2, 3, 9, 5])
    for i, t in enumerate((1, 2, 3, 4, 5, 6)):      # node 3 asks for 4, its child says 9
        logits[i, t] = 1.0
    step = api.VerifyStep(n, hq, hkv, d, 0, C + n, v, fmt="f16")
    step.run(cache, q, tk, tv, parent, tokens, logits)
    assert int(step.accept_len) == 4 and int(cache.ctx_len) == C + 4
    w = torch.zeros(hkv, C + n, device=DEV)
    api.kv_weights(cache, q, step.lse, w, path=step.path, accept_len=step.accept_len)
    total = w.double().sum(1).cpu().numpy()
    assert np.all(np.abs(total - 4 * 4) <= 16 * (2.0 ** -8))
    assert torch.all(w[:, :C + 4] > 0) and torch.all(w[:, C + 4:] == 0)


def test_equal_runs_streams_and_graphs():
    hkv, hq, d, C, n = 4, 24, 256, 5000, 9
    cache, _, q, lse, prev = make(8, hkv, d, C, C, "q4_0", n, hq)
    want = torch.empty(hkv, C, device=DEV)
    api.kv_weights(cache, q, lse, want, prev=prev)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty(hkv, C, device=DEV) for _ in range(4)]
    for i, o in enumerate(outs):
        api.kv_weights(cache, q, lse, o, prev=prev, stream=side[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    acc = prev.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.kv_weights(cache, q, lse, acc, prev=acc, decay=0.5)
    acc.copy_(prev)
    ref = prev.clone()
    for _ in range(3):
        g.replay()
        api.kv_weights(cache, q, lse, ref, prev=ref, decay=0.5)
    assert torch.equal(acc, ref)


def test_lengths_outside_the_cache():
    cache, _, q, lse, _ = make(1, 2, 64, 100, 100, "q4_0", 2, 4)
    want, out = torch.empty(2, 100, device=DEV), torch.empty(2, 100, device=DEV)
    api.kv_weights(cache, q, lse, want)
    for bad, same in ((101, True), (1 << 30, True), (-1, False)):
        cache.ctx_len.fill_(bad)
        out.fill_(-5.0)
        st = i32([0])
        api.kv_weights(cache, q, lse, out, status=st)
        assert int(st) == api.DEV_CTX
        assert torch.equal(out, want) if same else torch.all(out == -5.0)


def test_refusals():
    cache, _, q, lse, prev = make(1, 2, 64, 100, 100, "q4_0", 2, 4)
    out = torch.full((2, 100), -5.0, device=DEV)

    def no(c=cache, a=q, b=lse, o=out, **kw):
        with pytest.raises(api.DfvError):
            api.kv_weights(c, a, b, o, **kw)

    no(c=api.Int8Cache(2, 64, 100))
    no(a=q.float())
    no(a=q[0])
    no(a=q[:, :3].contiguous())                 # 3 query heads, 2 KV heads
    no(a=q[..., :32].contiguous())
    no(a=q.transpose(0, 1))
    no(b=lse.double())
    no(b=lse[:1].contiguous())
    no(o=out[:, :99].contiguous())
    no(o=out.double())
    no(prev=prev[:1].contiguous())
    no(prev=prev.cpu())
    no(window=-1)
    no(decay=math.nan)
    no(scale=math.nan)
    no(path=i32([0]))
    no(path=i32([0, 1]).long())
    no(accept_len=i32([]))
    assert torch.all(out == -5.0)
