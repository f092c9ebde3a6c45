"""Eviction by weight and rows read back, on the GPU: positions, bytes and
weights are equal to the plain selection's (``oracle/eviction.py``)."""

import math

import numpy as np
import pytest
import torch

import oracle.eviction as OV
from _helpers import DEV, need_gpu
from tree_verify_attention_gb300 import api
from test_gpu_kv_weights import i32, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def filled(seed, hkv, d, C, cap, fmt):
    g = torch.Generator().manual_seed(seed)
    cache = api.KVCache(hkv, d, cap, fmt=fmt)
    cache.k.copy_(torch.randint(0, 256, cache.k.shape, generator=g, dtype=torch.uint8))
    cache.v.copy_(torch.randint(0, 256, cache.v.shape, generator=g, dtype=torch.uint8))
    cache.ctx_len.fill_(C)
    w = torch.exp(2 * torch.randn(hkv, cap, generator=g))
    return cache, w.to(DEV)


def check(cache, w, keep, sinks=0, recent=0, dst_cap=None, dropped=0):
    hkv, cap, C = cache.n_kv_heads, cache.capacity, int(cache.ctx_len)
    dst_cap = dst_cap or keep
    into = api.KVCache(hkv, cache.head_dim, dst_cap, fmt=cache.fmt)
    into.k.fill_(171)
    into.v.fill_(172)
    cache.dropped.fill_(dropped)
    kept = torch.full((hkv, keep), -9, dtype=torch.int32, device=DEV)
    wo = torch.full((hkv, dst_cap), -5.0, device=DEV)
    st = i32([0])
    api.kv_evict(cache, w, into, kept, sinks=sinks, recent=recent, weights_out=wo, status=st)
    n = min(C, keep)
    assert int(st) == 0 and int(into.ctx_len) == n and int(into.dropped) == dropped + C - n
    wn = w.cpu().numpy()
    for h in range(hkv):
        want = OV.kept(wn[h, :C], keep, sinks, recent)
        assert kept[h, :n].tolist() == want
        at = torch.tensor(want, dtype=torch.long, device=DEV)
        assert torch.equal(into.k[h, :n], cache.k[h, at])
        assert torch.equal(into.v[h, :n], cache.v[h, at])
        assert np.array_equal(wo[h, :n].cpu().numpy(), wn[h, want], equal_nan=True)
    # what lies behind is left as it was
    assert torch.all(kept[:, n:] == -9) and torch.all(wo[:, n:] == -5.0)
    assert torch.all(into.k[:, n:] == 171) and torch.all(into.v[:, n:] == 172)
    return kept


@pytest.mark.parametrize("fmt", ["q4_0", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_shapes(fmt, d):
    for k, (hkv, C, cap, keep, s, r, dst) in enumerate((
            (1, 1, 1, 1, 0, 0, 1), (2, 100, 130, 10, 0, 0, 20), (3, 1001, 1001, 500, 4, 64, 501),
            (4, 4097, 5000, 2048, 4, 256, 2048), (8, 333, 400, 332, 1, 0, 400),
            (2, 50, 60, 50, 3, 3, 50), (2, 50, 60, 55, 20, 35, 60), (1, 0, 10, 5, 1, 1, 5),
            (5, 9000, 9001, 1, 0, 0, 1), (2, 700, 700, 12, 5, 7, 12), (2, 700, 700, 12, 12, 0, 13),
            (1, 40000, 40000, 19999, 100, 1000, 20000))):
        cache, w = filled(k, hkv, d, C, cap, fmt)
        check(cache, w, keep, s, r, dst, dropped=k * 10)


def test_long_caches():
    for hkv, C, keep in ((4, 131072, 32768), (1, 100003, 7), (2, 70001, 70000)):
        cache, w = filled(C, hkv, 64, C, C + 5, "q4_0")
        check(cache, w, keep, 3, 2)


def test_ties_and_special_weights():
    hkv, C = 3, 5000
    cache, w = filled(1, hkv, 64, C, C, "f16")
    g = torch.Generator().manual_seed(4)
    cases = [torch.zeros(hkv, C), torch.ones(hkv, C),
             torch.randint(0, 3, (hkv, C), generator=g).float(),
             -torch.randint(0, 3, (hkv, C), generator=g).float(),
             torch.randn(hkv, C, generator=g) * 1e-42,              # subnormal
             1.0 + torch.randint(0, 9, (hkv, C), generator=g).float() * 2.0 ** -23]
    odd = torch.randn(hkv, C, generator=g)
    odd[:, ::7], odd[:, 1::7], odd[:, 2::7] = math.nan, math.inf, -math.inf
    cases += [odd, torch.full((hkv, C), math.nan)]
    for x in cases:
        for keep, s, r in ((1, 0, 0), (777, 0, 0), (2500, 10, 10), (4999, 0, 1)):
            check(cache, x.to(DEV), keep, s, r)


def test_chained_evictions():
    """A cache cut twice: positions of the second cut go through the first's,
    dropped counts all rows that are gone."""
    cache, w = filled(3, 2, 128, 900, 1000, "q4_0")
    a, b = (api.KVCache(2, 128, c) for c in (400, 100))
    k1, k2 = i32(np.zeros((2, 400)).tolist()), i32(np.zeros((2, 100)).tolist())
    w1 = torch.zeros(2, 400, device=DEV)
    api.kv_evict(cache, w, a, k1, sinks=4, recent=16, weights_out=w1)
    api.kv_evict(a, w1, b, k2, sinks=4, recent=16)
    assert int(b.ctx_len) == 100 and int(b.dropped) == 800
    at = k1.long().gather(1, k2.long())
    for h in range(2):
        assert torch.equal(b.k[h], cache.k[h, at[h]]) and torch.equal(b.v[h], cache.v[h, at[h]])


def test_streams_and_graphs():
    cache, w = filled(5, 4, 256, 6000, 6000, "q4_0")
    want = check(cache, w, 1000, 4, 100)
    into = api.KVCache(4, 256, 1000)
    kept = torch.zeros(4, 1000, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    api.kv_evict(cache, w, into, kept, sinks=4, recent=100, stream=side)
    side.synchronize()
    assert torch.equal(kept, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.kv_evict(cache, w, into, kept, sinks=4, recent=100)
    for k in range(3):
        w.copy_(w.flip(1))
        cache.ctx_len.fill_(5000 - 100 * k)
        g.replay()
        n = 5000 - 100 * k
        for h in range(4):
            assert kept[h].tolist() == OV.kept(w[h, :n].cpu().numpy(), 1000, 4, 100)


def test_lengths_outside_the_cache():
    for bad, n in ((101, 50), (-3, 0)):
        cache, w = filled(6, 2, 64, 100, 100, "f16")
        cache.ctx_len.fill_(bad)
        into = api.KVCache(2, 64, 50, fmt="f16")
        st, kept = i32([0]), torch.zeros(2, 50, dtype=torch.int32, device=DEV)
        api.kv_evict(cache, w, into, kept, status=st)
        assert int(st) == api.DEV_CTX and int(into.ctx_len) == n


@pytest.mark.parametrize("fmt", ["q4_0", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_read(fmt, d):
    hkv, cap = 3, 301
    g = torch.Generator().manual_seed(d)
    cache = api.KVCache(hkv, d, cap, fmt=fmt)
    cache.fill(torch.randn(hkv, cap, d, generator=g).to(DEV),
               torch.randn(hkv, cap, d, generator=g).to(DEV))
    want = {w: torch.from_numpy(values(cache, cap, w)) for w in ("k", "v")}
    for pos, n in ((0, cap), (1, 300), (77, 5), (300, 1), (12, 0)):
        for dtype in (torch.float32, torch.bfloat16):
            for head_major in (False, True):
                shape = (hkv, n, d) if head_major else (n, hkv, d)
                wide = [torch.full(shape[:2] + (d + 8,), 7.0, dtype=dtype, device=DEV)
                        for _ in range(2)]
                out = [x[..., :d] for x in wide]
                cache.read(pos, n, *out, head_major=head_major)
                for o, x, w in zip(out, wide, ("k", "v")):
                    ref = want[w][:, pos:pos + n].to(dtype)     # (exact in float64: one rounding)
                    ref = ref if head_major else ref.transpose(0, 1)
                    assert torch.equal(o.cpu(), ref) and torch.all(x[..., d:] == 7.0)


def test_refusals():
    cache, w = filled(7, 2, 64, 100, 100, "q4_0")
    into = api.KVCache(2, 64, 50)
    kept = torch.full((2, 50), -9, dtype=torch.int32, device=DEV)

    def no(c=cache, a=w, i=into, k=kept, **kw):
        with pytest.raises(api.DfvError):
            api.kv_evict(c, a, i, k, **kw)

    no(c=api.Int8Cache(2, 64, 100))
    no(i=api.Int8Cache(2, 64, 100))
    no(i=cache)
    no(i=api.KVCache(2, 64, 50, fmt="f16"))
    no(i=api.KVCache(2, 128, 50))
    no(i=api.KVCache(3, 64, 50))
    no(a=w[:, :99].contiguous())
    no(a=w.double())
    no(k=kept.long())
    no(k=torch.zeros(2, 51, dtype=torch.int32, device=DEV))
    no(k=kept[:, :0])
    no(k=kept[0])
    no(sinks=-1)
    no(recent=-1)
    no(sinks=30, recent=21)
    no(weights_out=torch.zeros(2, 49, device=DEV))
    no(weights_out=w)
    assert torch.all(kept == -9) and not into.k.any() and int(into.ctx_len) == 0
    out = torch.zeros(5, 2, 64, device=DEV)
    for bad in ((96, 5, out, out), (-1, 5, out, out), (0, 5, out, out.bfloat16()),
                (0, 4, out, out), (0, 5, out, out.cpu()), (0, 5, out.half(), out.half())):
        with pytest.raises(api.DfvError):
            cache.read(*bad)
