"""Norm, rotation and values carried along on the GPU against the float64
definition (``oracle/encode.py``).

Tolerance of a float32 output that mixes a and b (both normed and weighted):
the sum of squares has a chain of 16 + 4 additions, halved by the root, then
root, quotient and two products: under 16 * 2^-24 relative in a and in b. The
angle is cut to 2^-32 of a turn and rounded to 24 bits (under 2^-22 rad
together), sine and cosine are within 2 units of 2^-24, product and sum add 2
roundings: under (16 + 4 + 2 + 2) 2^-24 (|a| + |b|). bf16 outputs add half a
step, 2^-8 of the value."""

import math

import numpy as np
import pytest
import torch

import oracle.encode as OE
from _helpers import DEV, need_gpu
from tree_verify_attention_gb300 import api

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def weights(d, seed=5):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.3 * torch.randn(2, d, generator=g)).to(DEV)


def rows(seed, n, heads, d, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, heads, d, generator=g) * scale).to(dtype).to(DEV)


def want_of(x, w, eps, pos, freq, near):
    x = x.double().cpu().numpy()
    y = x if eps is None else OE.norm(x, None if w is None else w.cpu().numpy(), eps)
    a = OE.rotate(y, pos, freq, near)
    # |a| + |b| of each output's pair
    m, half = np.abs(y), len(freq)
    both = m.copy()
    for i in range(half):
        p = (2 * i, 2 * i + 1) if near else (i, i + half)
        both[..., p[0]] = both[..., p[1]] = m[..., p[0]] + m[..., p[1]]
    return a, both


def near_enough(got, ref, both, dtype):
    got = got.double().cpu().numpy()
    tol = 24 * 2.0 ** -24 * both
    if dtype == BF16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) - tol)


def outs(n, hq, hkv, d, dtype):
    return [torch.full((n, h, d), 7.0, dtype=dtype, device=DEV) for h in (hq, hkv, hkv)]


def check(q, k, v, d, rot, near, pos, dst, place, eps=1e-6, w=None, base=1e6, out=None):
    n, hq, hkv = q.shape[0], q.shape[1], k.shape[1]
    rope = api.Rope(d, rot, base=base, interleaved=near, device=DEV)
    freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    src = [x.clone() for x in (q, k, v)]
    qo, ko, vo = out or outs(n, hq, hkv, d, dst)
    st = i32([0])
    api.qk_norm_rope(q, k, v, rope, qo, ko, vo, *(w if w is not None else (None, None)), eps=eps,
                     status=st, **place)
    for x, o, i in ((src[0], qo, 0), (src[1], ko, 1)):
        near_enough(o, *want_of(x, None if w is None else w[i], eps, pos, freq, near), dst)
    assert torch.equal(vo, src[2].to(dst))
    return int(st)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("src,dst", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
def test_types_and_rotated_parts(d, near, src, dst):
    for n, hq, hkv, rot in ((1, 24, 4, d), (3, 5, 1, d // 4), (70, 8, 8, d // 2), (2, 1, 3, 16)):
        pos = np.random.default_rng(n).integers(0, 1 << 20, n)
        q, k, v = (rows(n + i, n, h, d, src) for i, h in enumerate((hq, hkv, hkv)))
        check(q, k, v, d, rot, near, pos, dst, {"positions": i32(pos.tolist())}, w=weights(d))


@pytest.mark.parametrize("n", [1, 23, 65])
def test_tree_positions(n):
    d, hq, hkv = 256, 24, 4
    r = np.random.default_rng(n)
    parent = [-1] + [int(r.integers(0, i)) for i in range(1, n)]
    pos = 61440 + 1234 + OE.depths(parent)
    q, k, v = (rows(i, n, h, d, BF16) for i, h in enumerate((hq, hkv, hkv)))
    place = {"ctx_len": i32([61440]), "dropped": i32([1234]), "parent": i32(parent)}
    assert check(q, k, v, d, d, False, pos, BF16, place, w=weights(d)) == 0


def test_a_chain_of_all_nodes_and_bad_parents():
    n, d = 65, 64
    q, k, v = (rows(i, n, h, d, F32) for i, h in enumerate((2, 1, 1)))
    chain = [-1] + list(range(n - 1))
    place = {"ctx_len": i32([5]), "parent": i32(chain)}
    assert check(q, k, v, d, d, True, 5 + np.arange(n), F32, place) == 0
    bad = list(chain)
    bad[3], bad[40], bad[64] = 3, -2, 1 << 30       # taken as the root's children
    place["parent"] = i32(bad)
    assert check(q, k, v, d, d, True, 5 + OE.depths(bad), F32, place) == api.DEV_BAD_TREE


def test_rows_after_the_committed_length():
    n, d = 1000, 128
    q, k, v = (rows(i, n, h, d, BF16) for i, h in enumerate((4, 2, 2)))
    check(q, k, v, d, d, False, 777 + np.arange(n), BF16, {"ctx_len": i32([777])})


def test_far_and_negative_positions():
    """Angles of positions up to 2^31 - 1: the float64 product itself is off by
    2^31 * 2^-53 rad at most."""
    pos = [0, 1, (1 << 31) - 1, -1, -(1 << 31), 123456789, 131071]
    q, k, v = (rows(i, len(pos), 2, 64, F32) for i in range(3))
    check(q, k, v, 64, 64, False, pos, F32, {"positions": i32(pos)}, base=1e4)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_slices_of_a_projection_and_odd_strides(dtype):
    n, hq, hkv, d = 9, 6, 2, 128
    for pad, off in ((0, 0), (64, 0), (7, 3)):       # the last: rows on no boundary
        x = rows(3, n, 1, (hq + 2 * hkv) * d + pad, dtype)[:, 0]
        flat = torch.empty(x.numel() + off, dtype=dtype, device=DEV)[off:].view_as(x).copy_(x)
        q = flat[:, :hq * d].view(n, hq, d)
        k = flat[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
        v = flat[:, (hq + hkv) * d:(hq + 2 * hkv) * d].view(n, hkv, d)
        check(q, k, v, d, 64, True, np.arange(n), dtype, {"ctx_len": i32([0])}, w=weights(d))
    # heads before rows
    q, k, v = (rows(4 + i, h, n, d, dtype).transpose(0, 1) for i, h in enumerate((hq, hkv, hkv)))
    check(q, k, v, d, d, False, np.arange(n), dtype, {"ctx_len": i32([0])})


def test_in_place():
    n, d = 17, 256
    q, k, v = (rows(i, n, h, d, BF16) for i, h in enumerate((24, 4, 4)))
    check(q, k, v, d, 64, False, 100 + np.arange(n), BF16, {"ctx_len": i32([100])}, w=weights(d),
          out=(q, k, v))


def test_parts():
    """Without a norm, without a rotation, queries or keys alone, no rows."""
    n, d = 5, 128
    q, k, v = (rows(i, n, 2, d, F32) for i in range(3))
    check(q, k, v, d, d, False, np.arange(n), F32, {"ctx_len": i32([0])}, eps=None)
    check(q, k, v, d, 0, False, np.arange(n), F32, {"ctx_len": i32([0])}, w=weights(d))
    rope = api.Rope(d, device=DEV)
    both, alone = outs(n, 2, 2, d, F32), outs(n, 2, 2, d, F32)
    api.qk_norm_rope(q, k, v, rope, *both, ctx_len=i32([9]))
    api.qk_norm_rope(q, None, None, rope, alone[0], None, ctx_len=i32([9]))
    api.qk_norm_rope(None, k, None, rope, None, alone[1], ctx_len=i32([9]))
    assert torch.equal(both[0], alone[0]) and torch.equal(both[1], alone[1])
    assert torch.all(alone[2] == 7.0)
    api.qk_norm_rope(q[:0], k[:0], v[:0], rope, *(o[:0] for o in both), ctx_len=i32([9]))


def test_magnitudes():
    """Rows whose squares leave float32, or vanish in it, are normed all the same."""
    d = 64
    for scale in (1e30, 3e37, 1e-18, 1e-25, 1e-30):
        q, k, v = (rows(i, 4, 3, d, F32, scale) for i in range(3))
        for eps in (0.0, 1e-30):
            check(q, k, v, d, d, False, np.arange(4), F32, {"ctx_len": i32([0])}, eps=eps)
        check(q, k, v, d, d, False, np.arange(4), F32, {"ctx_len": i32([0])}, eps=1e-6)
    # a large head beside ordinary ones
    q = rows(7, 4, 3, d, F32)
    q[1, 1] *= 1e32
    check(q, k, v, d, d, True, np.arange(4), F32, {"ctx_len": i32([0])}, w=weights(d))


def test_infinities_and_nan_stay_in_their_head():
    d, n = 128, 6
    q, k, v = (rows(i, n, 4, d, BF16) for i in range(3))
    clean = outs(n, 4, 4, d, BF16)
    rope = api.Rope(d, device=DEV)
    api.qk_norm_rope(q, k, v, rope, *clean, ctx_len=i32([3]))
    q[2, 1, 5], q[4, 3, 100], k[0, 0, 0] = math.inf, math.nan, -math.inf
    v[1, 1, 1] = math.inf
    got = outs(n, 4, 4, d, BF16)
    api.qk_norm_rope(q, k, v, rope, *got, ctx_len=i32([3]))
    hit = torch.zeros(n, 4, dtype=torch.bool, device=DEV)
    hit[2, 1] = hit[4, 3] = True
    assert torch.equal(got[0][~hit], clean[0][~hit])
    assert torch.isnan(got[0][2, 1, 5]) and torch.isnan(got[0][2, 1, 5 + d // 2])
    assert torch.isnan(got[0][4, 3]).all()
    assert torch.equal(got[1][1:], clean[1][1:]) and torch.equal(got[1][0, 1:], clean[1][0, 1:])
    assert torch.equal(got[2], v)


def test_infinities_outside_the_rotated_part():
    """Dims that are not rotated do not meet: an infinity stays alone."""
    d, n = 256, 3
    for near in (False, True):
        q, k, v = (rows(i, n, 2, d, F32) for i in range(3))
        rope = api.Rope(d, 64, interleaved=near, device=DEV)
        clean, got = outs(n, 2, 2, d, F32), outs(n, 2, 2, d, F32)
        api.qk_norm_rope(q, k, v, rope, *clean, ctx_len=i32([3]), eps=None)
        q[1, 1, 200], k[0, 0, 65] = math.inf, -math.inf
        api.qk_norm_rope(q, k, v, rope, *got, ctx_len=i32([3]), eps=None)
        clean[0][1, 1, 200], clean[1][0, 0, 65] = math.inf, -math.inf
        assert all(torch.equal(a, b) for a, b in zip(got, clean))


def test_streams_and_graphs():
    n, d = 23, 256
    q, k, v = (rows(i, n, h, d, BF16) for i, h in enumerate((24, 4, 4)))
    rope, ctx = api.Rope(d, device=DEV), i32([1000])
    want = outs(n, 24, 4, d, BF16)
    api.qk_norm_rope(q, k, v, rope, *want, ctx_len=ctx)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = outs(n, 24, 4, d, BF16)
    api.qk_norm_rope(q, k, v, rope, *got, ctx_len=ctx, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    again = outs(n, 24, 4, d, BF16)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.qk_norm_rope(q, k, v, rope, *again, ctx_len=ctx)
    ctx.fill_(1000)
    q.copy_(q.flip(0))
    g.replay()
    api.qk_norm_rope(q, k, v, rope, *want, ctx_len=ctx)
    assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_refusals():
    d, n = 128, 4
    q, k, v = (rows(i, n, 2, d, BF16) for i in range(3))
    rope = api.Rope(d, device=DEV)
    o = outs(n, 2, 2, d, BF16)
    ctx = i32([0])

    def no(*a, **kw):
        with pytest.raises(api.DfvError):
            api.qk_norm_rope(*a, **kw)

    no(q, k, v, rope, *o)                                            # no place
    no(q, k, v, rope, *o, ctx_len=ctx, positions=i32([0] * n))
    no(q, k, v, rope, *o, positions=i32([0] * (n - 1)))
    no(q, k, v, rope, *o, ctx_len=ctx.long())
    no(q, k, v, rope, *o, ctx_len=ctx.cpu())
    no(q, k, v, api.Rope(64, device=DEV), *o, ctx_len=ctx)
    no(q, k, v, rope, o[0].float(), o[1], o[2], ctx_len=ctx)         # outputs of two types
    no(q, k.float(), v, rope, *o, ctx_len=ctx)
    no(q, k, v, rope, o[0][:, :1], o[1], o[2], ctx_len=ctx)
    no(q.transpose(1, 2), k, v, rope, *o, ctx_len=ctx)
    no(q, k, v.half(), rope, *o, ctx_len=ctx)
    no(q, None, v, rope, *o, ctx_len=ctx)
    no(None, None, None, rope, *o, ctx_len=ctx)
    no(q, k, v, rope, *o, ctx_len=ctx, eps=-1.0)
    no(q, k, v, rope, *o, ctx_len=ctx, eps=math.nan)
    no(q, k, v, rope, *o, weights(d)[0], ctx_len=ctx, eps=None)
    no(q, k, v, rope, *o, weights(64)[0], ctx_len=ctx)
    no(q, k, v, rope, *o, ctx_len=ctx, parent=i32([0] * (n - 1)))
    big = rows(0, 66, 2, d, BF16)
    no(big, big, big, rope, *outs(66, 2, 2, d, BF16), ctx_len=ctx, parent=i32([0] * 66))
    assert all(torch.all(x == 7.0) for x in o)
