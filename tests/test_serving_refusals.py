"""What the operators around a step refuse before any launch (CPU: no kernel is
reached): positions and norms, draws, and the weights and rows of a bounded
cache, at the C entries and in the binding."""

import ctypes
import math

import pytest
import torch

from test_int8_binding import OnDevice
from tree_verify_attention_gb300 import _lib, api
from tree_verify_attention_gb300 import build as B

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _lib.load()


# addresses that are never followed: every call below is refused on the host
A = 1 << 20


def encode(lib, n=5, hq=8, hkv=2, d=128, q=A, k=A, v=A, src=1, qw=A, kw=A, eps=1e-6, turns=A,
           rot=64, near=0, pos=None, par=A, ctx=A, dropped=A, qo=A, ko=A, vo=A, dst=1):
    return lib.dfv_qk_norm_rope(n, hq, hkv, d, q, k, v, src, 1024, d, 256, d, 256, d, qw, kw, eps,
                                turns, rot, near, pos, par, ctx, dropped, qo, ko, vo, dst, None,
                                None)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=(1 << 26) + 1, par=None), dict(hq=-1), dict(hkv=-1), dict(hq=1025),
    dict(hkv=1025), dict(hq=0, hkv=0, q=None, k=None, v=None), dict(rot=-16), dict(rot=8),
    dict(rot=144), dict(eps=math.nan), dict(n=66), dict(q=None), dict(k=None), dict(qo=None),
    dict(ko=None), dict(vo=None), dict(hkv=0, k=None), dict(turns=None), dict(ctx=None, par=None),
    dict(pos=A), dict(pos=A, ctx=None, dropped=None), dict(pos=A, par=None, dropped=None),
    dict(pos=A, par=None, ctx=None), dict(eps=-1.0), dict(eps=-1.0, kw=None), dict(q=A + 1),
    dict(k=A + 1), dict(v=A + 1), dict(src=0, q=A + 2), dict(qo=A + 8), dict(ko=A + 8),
    dict(vo=A + 8), dict(qw=A + 4), dict(kw=A + 4), dict(turns=A + 4), dict(par=A + 2),
    dict(ctx=A + 2), dict(dropped=A + 2), dict(pos=A + 2, par=None, ctx=None, dropped=None)],
    ids=str)
def test_encode(lib, kw):
    assert encode(lib, **kw) == INVALID


def test_encode_kinds(lib):
    for kw in (dict(d=32), dict(d=96), dict(d=512), dict(d=0), dict(src=2), dict(src=-1),
               dict(dst=2)):
        assert encode(lib, **kw) == UNSUPPORTED
    assert encode(lib, n=0) == OK


def sampling(**kw):
    f = dict(temperature=None, top_k=None, top_p=None, min_p=None, temperature_all=1.0,
             top_k_all=0, top_p_all=1.0, min_p_all=0.0)
    f.update(kw)
    return _lib.SamplingStruct(**f)


def sample(lib, n=5, v=1000, dt=1, x=A, stride=1000, u=A, s=sampling(), tok=A, lp=A):
    return lib.dfv_sample(n, v, dt, x, stride, u, ctypes.addressof(s) if s else None, tok, lp,
                          None, None)


def accept(lib, n=5, v=1000, dt=1, x=A, stride=1000, u=A, s=sampling(), tok=A, lp=A, par=A,
           tokens=A, al=A, path=A, out=A, ws=A, ws_bytes=256):
    return lib.dfv_sample_accept(n, v, dt, x, stride, u, ctypes.addressof(s) if s else None, par,
                                 tokens, tok, lp, al, path, out, ws, ws_bytes, None, None)


@pytest.mark.parametrize("call", [sample, accept])
@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=(1 << 26) + 1), dict(v=0), dict(v=-5), dict(stride=999), dict(stride=-1000),
    dict(x=None), dict(u=None), dict(s=None), dict(tok=None), dict(x=A + 1), dict(dt=0, x=A + 2),
    dict(u=A + 2), dict(tok=A + 2), dict(lp=A + 2), dict(s=sampling(temperature=A + 2)),
    dict(s=sampling(top_k=A + 1)), dict(s=sampling(top_p=A + 2)), dict(s=sampling(min_p=A + 3))],
    ids=str)
def test_sample(lib, call, kw):
    assert call(lib, **kw) == INVALID


def test_sample_kinds(lib):
    for call in (sample, accept):
        assert call(lib, dt=2) == UNSUPPORTED
        assert call(lib, v=(1 << 19) + 1, stride=1 << 20) == UNSUPPORTED
    assert sample(lib, n=0) == OK


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(n=66), dict(par=None), dict(tokens=None), dict(al=None), dict(path=None),
    dict(out=None), dict(ws=None), dict(par=A + 2), dict(tokens=A + 2), dict(al=A + 2),
    dict(path=A + 2), dict(out=A + 2), dict(ws=A + 128)], ids=str)
def test_accept(lib, kw):
    assert accept(lib, **kw) == INVALID


def test_accept_workspace(lib):
    assert accept(lib, ws_bytes=255) == WORKSPACE
    need = lib.dfv_sample_accept_workspace_bytes
    assert need(5, 1000) == 256 and need(65, 1 << 19) == 256
    for n, v in ((0, 1000), (66, 1000), (5, 0), (5, (1 << 19) + 1), (-1, 5)):
        assert need(n, v) == 0


def weights(lib, n=5, hq=8, hkv=2, d=128, window=0, fmt=2, cap=1000, ctx=A, k=A, q=A, lse=A,
            path=A, al=A, scale=0.0, decay=1.0, prev=A, w=A):
    return lib.dfv_kv_weights(n, hq, hkv, d, window, fmt, cap, ctx, k, q, lse, path, al, scale,
                              decay, prev, w, None, None)


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(n=-1), dict(n=65537), dict(hkv=0), dict(hq=1), dict(hq=9), dict(hq=1026),
    dict(window=-1), dict(cap=0), dict(cap=(1 << 30) + 1), dict(scale=math.nan),
    dict(decay=math.nan), dict(ctx=None), dict(k=None), dict(q=None), dict(lse=None), dict(w=None),
    dict(k=A + 8), dict(q=A + 8), dict(lse=A + 2), dict(prev=A + 2), dict(w=A + 2),
    dict(ctx=A + 2), dict(path=A + 2), dict(al=A + 2)], ids=str)
def test_weights(lib, kw):
    assert weights(lib, **kw) == INVALID


def evict(lib, hkv=2, d=128, fmt=2, cap=1000, ctx=A, dropped=A, k=A, v=2 * A, w=A, keep=100,
          sinks=4, recent=20, dst_cap=200, kd=3 * A, vd=4 * A, dctx=2 * A, ddrop=A, wo=2 * A,
          kept=A):
    return lib.dfv_kv_evict(hkv, d, fmt, cap, ctx, dropped, k, v, w, keep, sinks, recent, dst_cap,
                            kd, vd, dctx, ddrop, wo, kept, None, None)


@pytest.mark.parametrize("kw", [
    dict(hkv=0), dict(hkv=65536), dict(cap=0), dict(cap=(1 << 30) + 1), dict(keep=0),
    dict(keep=201), dict(dst_cap=(1 << 30) + 1), dict(sinks=-1), dict(recent=-1), dict(sinks=81),
    dict(sinks=(1 << 31) - 1, recent=(1 << 31) - 1), dict(ctx=None), dict(k=None), dict(v=None),
    dict(w=None), dict(kd=None), dict(vd=None), dict(dctx=None), dict(kept=None), dict(k=A + 8),
    dict(v=A + 8), dict(kd=A + 8), dict(vd=A + 8), dict(w=A + 2), dict(wo=A + 2), dict(kept=A + 2),
    dict(ctx=A + 2), dict(dctx=A + 2), dict(dropped=A + 2), dict(ddrop=A + 2), dict(kd=A),
    dict(vd=2 * A), dict(kd=2 * A), dict(vd=A), dict(vd=3 * A), dict(dctx=A), dict(wo=A)], ids=str)
def test_evict(lib, kw):
    assert evict(lib, **kw) == INVALID


def read(lib, hkv=2, d=128, fmt=2, cap=1000, pos=0, n=5, k=A, v=A, kd=A, vd=A, dst=1):
    return lib.dfv_kv_read_rows(hkv, d, fmt, cap, pos, n, k, v, kd, vd, dst, 256, 128, None)


@pytest.mark.parametrize("kw", [
    dict(hkv=0), dict(hkv=65536), dict(cap=0), dict(pos=-1), dict(n=-1), dict(pos=996),
    dict(pos=(1 << 31) - 1, n=(1 << 31) - 1), dict(k=None), dict(v=None), dict(kd=None),
    dict(vd=None), dict(k=A + 8), dict(v=A + 8), dict(kd=A + 1), dict(dst=0, vd=A + 2)], ids=str)
def test_read(lib, kw):
    assert read(lib, **kw) == INVALID


def test_kinds(lib):
    for call in (weights, evict, read):
        for kw in (dict(d=32), dict(d=96), dict(d=512), dict(fmt=3), dict(fmt=-1),
                   dict(fmt=1 << 8)):
            assert call(lib, **kw) == UNSUPPORTED
    assert read(lib, dst=2) == UNSUPPORTED
    assert read(lib, n=0) == OK


# ---- the binding's own checks

def cpu_cache(capacity=200, fmt="q4_0"):
    return api.KVCache(2, 64, capacity, device="cpu", fmt=fmt)


@pytest.mark.parametrize("kw", [
    dict(temperature=-1.0), dict(temperature=math.inf), dict(temperature=math.nan),
    dict(top_p=math.nan), dict(min_p=math.nan), dict(top_k=math.nan),
    dict(temperature=torch.ones(3)), dict(top_k=torch.ones(3))], ids=str)
def test_sampling_parameters(kw):
    with pytest.raises(api.DfvError):
        api.Sampling(**kw)


@pytest.mark.parametrize("k,want", [(1 << 31, 2 ** 31 - 1), (1 << 32, 2 ** 31 - 1), (-5, 0),
                                    (math.inf, 2 ** 31 - 1), (-math.inf, 0), (7, 7)])
def test_top_k_is_clamped(k, want):
    assert api.Sampling(top_k=k)._struct.top_k_all == want


def test_rows_longer_than_any_vocabulary():
    x = OnDevice(torch.zeros(1, 1).expand(1, (1 << 32) + 7))
    x.stride = lambda: ((1 << 32) + 7, 1)
    with pytest.raises(api.DfvError, match="at most"):
        api.sample_tokens(x, None, api.Sampling(), None)


@pytest.mark.parametrize("window", [-1, 1 << 31, 1 << 32])
def test_windows_of_the_weights(window):
    c, q = cpu_cache(), OnDevice(torch.zeros(3, 4, 64, dtype=torch.bfloat16))
    with pytest.raises(api.DfvError, match="window"):
        api.kv_weights(c, q, torch.zeros(3, 4), torch.zeros(2, 200), window=window)


def test_caches_of_an_eviction():
    c, w, kept = cpu_cache(), torch.zeros(2, 200), torch.zeros(2, 50, dtype=torch.int32)
    for into in (c, cpu_cache(fmt="f16"), api.KVCache(2, 128, 200, device="cpu"),
                 api.KVCache(3, 64, 200, device="cpu"), api.Int8Cache(2, 64, 200, device="cpu")):
        with pytest.raises(api.DfvError):
            api.kv_evict(c, w, into, kept)
    with pytest.raises(api.DfvError):
        api.kv_evict(api.Int8Cache(2, 64, 200, device="cpu"), w, c, kept)


def test_rows_outside_a_cache():
    c, out = cpu_cache(), torch.zeros(3, 2, 64)
    for pos, n in ((-1, 3), (198, 3), (0, 201), (0, -1), (5, 1 << 32), (1 << 32, 3)):
        with pytest.raises(api.DfvError, match="outside"):
            c.read(pos, n, out, out)


def test_a_step_takes_random_numbers_only_if_it_draws():
    step = object.__new__(api.VerifyStep)      # (a step's buffers need a GPU)
    step.shape, step.int8 = (4, 6, 2, 64, 0, 200, 50), False
    for s, u in ((None, torch.zeros(4)), (api.Sampling(), None)):
        step.sampling = s
        with pytest.raises(api.DfvError, match="uniform"):
            step.run(cpu_cache(), None, None, None, None, None, None, uniform=u)


def test_rope():
    for kw in (dict(head_dim=96), dict(head_dim=64, rot_dim=8), dict(head_dim=64, rot_dim=80),
               dict(head_dim=64, rot_dim=-16), dict(head_dim=64, inv_freq=[1.0] * 31),
               dict(head_dim=64, inv_freq=[math.inf] * 32),
               dict(head_dim=64, inv_freq=[math.nan] * 32)):
        with pytest.raises(api.DfvError):
            api.Rope(device="cpu", **kw)
