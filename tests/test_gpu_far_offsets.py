"""Caches, logits and rows whose offsets pass 2^32 bytes and 2^31 elements."""

import math

import numpy as np
import pytest
import torch

import oracle
from _helpers import DEV, need_gpu
from tree_verify_attention_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def long_cache(fmt):
    hkv, d, cap = (8, 256, 1_100_003) if fmt == "f16" else (16, 256, 1_900_003)
    cache = api.KVCache(hkv, d, cap, fmt=fmt)
    torch.manual_seed(3)
    for t in (cache.k, cache.v):
        if fmt == "f16":
            t.view(torch.float16).normal_()
            continue
        t.random_(0, 256)
        scale = (0.05 + 0.2 * torch.rand(hkv, cap, d // 32, 1, device=DEV)).half()
        t.view(hkv, cap, d // 32, 18)[..., :2] = scale.view(torch.uint8)
    assert cache.k.numel() > 1 << 32
    cache.ctx_len.fill_(cap - 2)
    return cache


def rows_of(cache, which, h, at):
    b = getattr(cache, which)[h, at].cpu().numpy()
    if cache.fmt == "f16":
        return b.view(np.float16).astype(np.float64)
    return oracle.q4_0.dequantize_rows(b.reshape(len(b), -1, 18)).astype(np.float64)


@pytest.mark.parametrize("fmt", ["q4_0", "f16"])
def test_caches(fmt):
    cache = long_cache(fmt)
    hkv, d, cap = cache.n_kv_heads, cache.head_dim, cache.capacity
    C, n, hq = cap - 2, 3, 2 * hkv
    g = torch.Generator().manual_seed(4)
    at = torch.cat([torch.randint(0, C, (500,), generator=g),
                    torch.tensor([0, C - 4, C - 3, C - 2, C - 1])])
    # weights (the tolerance of a term as in the operator's own tests)
    q = (0.3 * torch.randn(n, hq, d, generator=g)).to(torch.bfloat16)
    lse = 1 + torch.rand(n, hq, generator=g)
    w = torch.full((hkv, cap), -5.0, device=DEV)
    st = i32([0])
    api.kv_weights(cache, q.to(DEV), lse.to(DEV), w, status=st)
    qd, ld, scale = q.double().numpy(), lse.double().numpy(), 1 / math.sqrt(d)
    for h in range(hkv):
        k = rows_of(cache, "k", h, at.to(DEV))
        ref, tol = np.zeros(len(at)), np.zeros(len(at))
        for s in range(n):
            sees = at.numpy() <= C - n + s
            for hh in (2 * h, 2 * h + 1):
                x, a = scale * (k @ qd[s, hh]), scale * (np.abs(k) @ np.abs(qd[s, hh]))
                term = np.where(sees, np.exp(x - ld[s, hh]), 0)
                ref += term
                tol += term * (d / 8 * 2.0 ** -23 * a + 2.0 ** -22 * (np.abs(x) + ld[s, hh])
                               + 2.0 ** -21)
        tol += (n * 2 + 8) * 2.0 ** -24 * ref
        assert np.all(np.abs(w[h, at].double().cpu().numpy() - ref) <= tol)
    assert torch.all(w[:, C:] == -5.0) and int(st) == 0
    # eviction by distinct weights
    for h in range(hkv):
        w[h] = torch.randperm(cap, device=DEV).float()
    keep, sinks, recent = 4099, 4, 16
    into = api.KVCache(hkv, d, keep, fmt=fmt)
    kept = torch.empty(hkv, keep, dtype=torch.int32, device=DEV)
    api.kv_evict(cache, w, into, kept, sinks=sinks, recent=recent, status=st)
    assert int(into.ctx_len) == keep and int(into.dropped) == C - keep and int(st) == 0
    for h in range(hkv):
        best = w[h, sinks:C - recent].topk(keep - sinks - recent).indices + sinks
        ends = torch.arange(C, device=DEV)
        want = torch.cat([ends[:sinks], best, ends[-recent:]]).sort().values
        assert torch.equal(kept[h].long(), want)
        assert torch.equal(into.k[h], cache.k[h, want])
        assert torch.equal(into.v[h], cache.v[h, want])
    # the last rows, beyond the committed length too
    ko, vo = (torch.empty(9, hkv, d, device=DEV) for _ in range(2))
    cache.read(cap - 9, 9, ko, vo)
    last = torch.arange(cap - 9, cap, device=DEV)
    for h in range(hkv):
        assert np.array_equal(ko[:, h].double().cpu().numpy(), rows_of(cache, "k", h, last))
        assert np.array_equal(vo[:, h].double().cpu().numpy(), rows_of(cache, "v", h, last))


def test_rows_far_apart():
    n, far = 40, 1 << 27
    store = torch.empty((n - 1) * far + 4096, dtype=torch.bfloat16, device=DEV)
    assert store.numel() > 1 << 32
    torch.manual_seed(5)
    x, u = (3 * torch.randn(n, 4000, device=DEV)).to(torch.bfloat16), torch.rand(n, device=DEV)
    rows = store.as_strided((n, 4000), (far, 1))
    rows.copy_(x)
    tok = [torch.empty(n, dtype=torch.int32, device=DEV) for _ in range(2)]
    for s in (api.Sampling(), api.Sampling(top_p=0.9), api.Sampling(top_k=20)):
        for a, t in ((x, tok[0]), (rows, tok[1])):
            api.sample_tokens(a, u, s, t)
        assert torch.equal(*tok)
    q = torch.randn(n, 8, 256, device=DEV).to(torch.bfloat16)
    heads = store.as_strided((n, 8, 256), (far, 256, 1))
    heads.copy_(q)
    rope, pos = api.Rope(256), torch.arange(n, dtype=torch.int32, device=DEV)
    out = [torch.empty_like(q) for _ in range(2)]
    for a, o in ((q, out[0]), (heads, out[1])):
        api.qk_norm_rope(a, None, None, rope, o, None, positions=pos)
    assert torch.equal(*out)


def test_many_rows():
    """Outputs beyond 2^31 elements; in place."""
    n, hq, d = 66_003, 128, 256
    q = torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV).normal_()
    assert q.numel() > 1 << 31
    rope, pos = api.Rope(d), torch.arange(n, dtype=torch.int32, device=DEV)
    some = torch.tensor([0, 1, 65535, 65536, n - 2, n - 1], device=DEV)
    src, want = q[some].contiguous(), torch.empty(6, hq, d, dtype=torch.bfloat16, device=DEV)
    api.qk_norm_rope(src, None, None, rope, want, None, positions=pos[some])
    api.qk_norm_rope(q, None, None, rope, q, None, positions=pos)
    assert torch.equal(q[some], want)
