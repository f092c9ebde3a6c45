"""What the 8-bit cache, its attention and the token log probabilities refuse
before any launch (CPU: no kernel is reached), and the oracle's 8-bit rule on
hand-made blocks."""

import ctypes

import numpy as np
import pytest
import torch

import oracle.int8 as I8
import oracle.logprobs as OL
from tree_verify_attention_gb300 import _lib, api
from tree_verify_attention_gb300 import build as B

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _lib.load()


# addresses that are never followed: every call below is refused on the host
A = 1 << 20


def cache(**kw):
    f = dict(n_kv_heads=4, head_dim=256, capacity=1000, reserved=0, state=A, k_codes=A, v_codes=A,
             k_scale=A, v_scale=A, k_tail=A, v_tail=A)
    f.update(kw)
    return _lib.Kv8CacheStruct(**f)


BAD_CACHES = [dict(n_kv_heads=0), dict(n_kv_heads=70000), dict(capacity=0),
              dict(capacity=(1 << 30) + 1), dict(state=None), dict(k_codes=None),
              dict(v_codes=None), dict(k_scale=None), dict(v_scale=None), dict(k_tail=None),
              dict(v_tail=None), dict(k_codes=A + 64), dict(v_codes=A + 16), dict(k_tail=A + 8),
              dict(v_scale=A + 2),
              dict(k_tail=A + 16), dict(v_tail=A + 16)]


def append(lib, c, at=0, n=5, k=A, v=A, dt=1):
    return lib.dfv_kv8_append(ctypes.addressof(c) if c else None, at, n, k, v, dt, 1024, 256, 1024,
                              256, None, None)


def commit(lib, c, n=23, L=A, path=A, k=A, v=A):
    return lib.dfv_kv8_commit(ctypes.addressof(c) if c else None, n, L, path, k, v, None, None)


def read(lib, c, pos=0, n=5, k=A, v=A, dt=1):
    return lib.dfv_kv8_read(ctypes.addressof(c) if c else None, pos, n, k, v, dt, 1024, 256, None,
                            None)


def attn(lib, c, n=23, md=16, hq=24, w=0, q=A, tk=A, tv=A, par=A, out=A, dt=1, ws=A,
         ws_bytes=1 << 40):
    return lib.dfv_kv8_attn(ctypes.addressof(c) if c else None, n, md, hq, w, q, tk, tv, par, 0.0,
                            out, dt, None, ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw", BAD_CACHES, ids=str)
def test_bad_caches(lib, kw):
    c = cache(**kw)
    for call in (append, commit, read, attn):
        assert call(lib, c) == INVALID
        assert call(lib, None) == INVALID


def test_bad_shapes_and_pointers(lib):
    c = cache()
    for d in (0, 32, 96, 512):
        for call in (append, commit, read, attn):
            assert call(lib, cache(head_dim=d)) == UNSUPPORTED
    assert append(lib, c, dt=2) == UNSUPPORTED and read(lib, c, dt=7) == UNSUPPORTED
    assert attn(lib, c, dt=2) == UNSUPPORTED
    for kw in (dict(at=-2), dict(n=-1), dict(n=1001), dict(at=996), dict(k=None), dict(v=None),
               dict(k=A + 1), dict(dt=0, v=A + 2)):
        assert append(lib, c, **kw) == INVALID, kw
    for kw in (dict(n=0), dict(n=66), dict(L=None), dict(path=None), dict(k=None), dict(v=A + 8)):
        assert commit(lib, c, **kw) == INVALID, kw
    for kw in (dict(pos=-1), dict(n=-1), dict(pos=996), dict(k=None), dict(v=A + 1)):
        assert read(lib, c, **kw) == INVALID, kw
    for kw in (dict(n=0), dict(n=66), dict(md=-1), dict(hq=0), dict(hq=25), dict(hq=260),
               dict(w=-1), dict(q=None), dict(tk=None), dict(tv=A + 8), dict(par=None),
               dict(out=None), dict(out=A + 4), dict(ws=None), dict(ws=A + 128)):
        assert attn(lib, c, **kw) == INVALID, kw
    assert attn(lib, c, ws_bytes=256) == WORKSPACE
    assert append(lib, c, at=-1, n=0, k=None, v=None) == 0
    assert read(lib, c, n=0, k=None, v=None) == 0


def test_workspace_sizes(lib):
    f = lib.dfv_kv8_attn_workspace_bytes
    assert f(23, 24, 4, 256, 2048, 61463) > 0
    for args in ((0, 24, 4, 256, 0, 10), (66, 24, 4, 256, 0, 10), (5, 24, 5, 256, 0, 10),
                 (5, 24, 4, 96, 0, 10), (5, 24, 4, 256, -1, 10), (5, 24, 4, 256, 0, 0),
                 (5, 260, 4, 256, 0, 10)):
        assert f(*args) == 0, args


def test_logprob_refusals(lib):
    def call(n=3, v=100, dt=1, x=A, st=100, tok=A, top=5, lp=A, e=A, ids=A, tl=A):
        return lib.dfv_token_logprobs(n, v, dt, x, st, tok, top, lp, e, ids, tl, None, None)

    assert call(dt=2) == UNSUPPORTED
    for kw in (dict(n=-1), dict(v=0), dict(x=None), dict(st=99), dict(tok=None), dict(top=-1),
               dict(top=33), dict(v=4, st=4), dict(ids=None, tl=None), dict(x=A + 1),
               dict(dt=0, x=A + 2)):
        assert call(**kw) == INVALID, kw
    assert call(n=0, x=None) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(2, 10)
    with pytest.raises(api.DfvError, match="CUDA"):
        api.token_logprobs(x, torch.zeros(2, dtype=torch.int32), torch.zeros(2))
    with pytest.raises(api.DfvError, match="head_dim"):
        api.Int8Cache(2, 96, 10, device="cpu")
    with pytest.raises(api.DfvError, match="shape"):
        api.Int8Cache(0, 64, 10, device="cpu")
    c = api.Int8Cache(2, 64, 10, device="cpu")
    assert c.k.shape == (2, 1, 4, 64, 16) and c.v.shape == (2, 1, 4, 64, 16)
    with pytest.raises(api.DfvError, match="CUDA"):
        c.append(torch.zeros(3, 2, 64), torch.zeros(3, 2, 64))
    with pytest.raises(api.DfvError, match="CUDA"):
        c.read(0, 3, torch.zeros(3, 2, 64), torch.zeros(3, 2, 64))
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    for kw in (dict(tree_as_cache=True), dict(pipelined=True)):
        with pytest.raises(api.DfvError, match="not available"):
            api.tree_verify_attn(c, q, q, q, None, 0, 1, None, None, None, **kw)
    with pytest.raises(api.DfvError, match="CUDA"):
        api.tree_verify_attn(c, q, q, q, torch.zeros(1, dtype=torch.int32), 0, 1, q, None, None)


def test_constants_match_the_header(lib):
    import re
    text = open(B.INCLUDE + "/dfv.h").read()
    defs = {m.group(1): int(m.group(2), 0)
            for m in re.finditer(r"#define\s+(DFV_\w+)\s+(0x[0-9a-fA-F]+|\d+)u?\b", text)}
    assert defs["DFV_DEV_NONFINITE"] == api.DEV_NONFINITE
    assert defs["DFV_DEV_BAD_TOKEN"] == api.DEV_BAD_TOKEN
    assert defs["DFV_MAX_TOP"] == api.MAX_TOP


def test_oracle_rule_by_hand():
    """One block with amax = 254: code = round-half-even(x / 2), scale 2."""
    x = np.zeros((1, 130, 64))
    x[0, 0, 0] = -254.0
    x[0, 1, :8] = [1, 3, 5, -1, -3, 253, 251, 0.98]
    x[0, 64, 0] = 2.0 ** -41
    x[0, 129, 5] = 0.3
    codes, scale = I8.encode_blocks(x)
    assert codes.shape == (1, 2, 64, 64) and codes[0, 0, 0, 0] == -127
    assert codes[0, 0, 1, :8].tolist() == [0, 2, 2, 0, -2, 126, 126, 0]
    assert scale.tolist() == [[2.0, 0.0]] and not codes[0, 1].any()
    v = I8.cached_values(x)
    assert v[0, 1, 1] == 4.0 and v[0, 64, 0] == 0.0 and v[0, 129, 5] == 0.3
    # the layouts of the header
    k = np.arange(4 * 64 * 16).reshape(1, 1, 4, 64, 16)
    assert I8.unpack_k(k)[0, 0, 5, 37] == k[0, 0, 2, 5, 5]
    v = np.arange(4 * 64 * 16).reshape(1, 1, 4, 64, 16)
    assert I8.unpack_v(v)[0, 0, 37, 5] == v[0, 0, 2, 5, 5]


def test_oracle_logprobs_by_hand():
    x = np.log(np.array([[1.0, 2.0, 5.0, 2.0], [1.0, 0.0 + 1e-300, 0.0 + 1e-300, 1.0]]))
    x[1, 1:3] = -np.inf
    lp, ent, ids, tlp = OL.token_logprobs(x, np.array([1, 0]), 4)
    assert np.allclose(lp, np.log([0.2, 0.5]))
    p = np.array([0.1, 0.2, 0.5, 0.2])
    assert np.allclose(ent, [-(p * np.log(p)).sum(), np.log(2)])
    assert ids.tolist() == [[2, 1, 3, 0], [0, 3, 1, 2]]
    assert np.allclose(tlp[0], np.log([0.5, 0.2, 0.2, 0.1])) and tlp[1, 2] == -np.inf
