"""Weights of keys for more query rows than one slice or one tile of scores
holds, and for rows of different magnitudes (the tolerance of
``test_gpu_kv_weights.py``)."""

import math

import numpy as np
import pytest
import torch

import oracle.eviction as OV
from _helpers import DEV, need_gpu
from test_gpu_kv_weights import check, i32, make, tolerance
from tree_verify_attention_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("fmt", ["f16", "q4_0"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hkv,hq,n", [(1, 8, 16), (2, 16, 17), (2, 8, 64), (1, 4, 65), (1, 8, 36),
                                      (1, 8, 37), (2, 16, 65)])
def test_rows_about_the_slices(fmt, d, hkv, hq, n):
    check(300 + n + d, hkv, hq, d, 1500 + n, fmt, n, decay=0.75, window=(0, 700)[n & 1])


@pytest.mark.parametrize("d", [64, 128])
def test_many_chunks_and_slices(d):
    """Each CTA has several chunks of more than one head."""
    check(77 + d, 8, 32, d, 30011, "f16", 65)


@pytest.mark.parametrize("fmt", ["f16", "q4_0"])
@pytest.mark.parametrize("first", [0, -30, 30])
@pytest.mark.parametrize("spread", [3, 8, 9, 12, 40])
def test_rows_of_different_magnitudes(fmt, first, spread):
    """Rows 2^0 to 2^spread apart, the first of them the largest, the smallest or
    another; scores stay moderate, as ``scale`` and the rows' own sizes cancel."""
    hkv, hq, d, C, n = 2, 8, 128, 700, 33
    cache, k, q, _, prev = make(5, hkv, d, C, C + 3, fmt, n, hq)
    e = torch.arange(n) * spread // (n - 1)
    e = e if first < 0 else spread - e if first > 0 else (e + spread // 2) % (spread + 1)
    q = (q.cpu().double() * 2.0 ** -(e.double())[:, None, None]).to(torch.bfloat16).to(DEV)
    scale = 1 / math.sqrt(d)
    qd = q.double().cpu().numpy()
    lse = np.zeros((n, hq))
    for h in range(hq):
        x = scale * qd[:, h] @ k[h // (hq // hkv)].T
        lse[:, h] = np.log(np.exp(x).sum(1))
    lse = torch.from_numpy(lse).float().to(DEV)
    out, st = torch.empty(hkv, C + 3, device=DEV), i32([0])
    api.kv_weights(cache, q, lse, out, status=st)
    ln = lse.double().cpu().numpy()
    ref = OV.weights(qd, ln, k, None)
    tol = tolerance(qd, ln, k, np.zeros((hkv, C)), 0, scale, d, ref)
    got = out.double().cpu().numpy()[:, :C]
    assert int(st) == 0
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)


@pytest.mark.parametrize("fmt", ["f16", "q4_0"])
@pytest.mark.parametrize("row", [0.0, math.nan, math.inf])
def test_a_first_row_without_a_magnitude(fmt, row):
    """It sets no exponent for the others."""
    hkv, hq, d, C, n = 2, 8, 128, 300, 20
    cache, k, q, lse, _ = make(6, hkv, d, C, C, fmt, n, hq)
    q[0] = row
    out, st = torch.empty(hkv, C, device=DEV), i32([0])
    api.kv_weights(cache, q, lse, out, status=st)
    qd, ln = q.double().cpu().numpy(), lse.double().cpu().numpy()
    ref = OV.weights(qd, ln, k, None)
    tol = tolerance(qd, ln, k, np.zeros((hkv, C)), 0, 1 / math.sqrt(d), d, ref)
    got = out.double().cpu().numpy()
    assert int(st) == (0 if row == 0 else api.DEV_NONFINITE)
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)


@pytest.mark.parametrize("fmt", ["f16", "q4_0"])
@pytest.mark.parametrize("window", [1, 4, 299, 300, 301, (1 << 31) - 1])
def test_windows_about_the_capacity(fmt, window):
    """Also with more rows than keys, whose first ones stand before position 0."""
    for C, n in ((5, 12), (300, 7)):
        check(8 + C, 2, 4, 64, C, fmt, n, cap=300, window=window)
