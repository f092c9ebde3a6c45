"""Pins of the oracle of key weights and eviction: closed forms and plain loops."""

import math

import numpy as np
import pytest

import oracle.eviction as OV


def test_weights_of_a_softmax_sum_to_one():
    r = np.random.default_rng(0)
    n, hq, hkv, d, C = 5, 6, 2, 8, 40
    q, k = r.standard_normal((n, hq, d)), r.standard_normal((hkv, C, d))
    lse = np.zeros((n, hq))
    for s in range(n):
        for h in range(hq):
            x = k[h // 3, :C - n + s + 1] @ q[s, h] / math.sqrt(d)
            lse[s, h] = np.log(np.exp(x).sum())
    w = OV.weights(q, lse, k, None)
    assert np.allclose(w.sum(1), n * 3)             # each row and head gives 1
    assert np.allclose(w[:, -1], [sum(math.exp(k[g, -1] @ q[-1, h] / math.sqrt(d) - lse[-1, h])
                                      for h in range(3 * g, 3 * g + 3)) for g in range(2)])


def test_weights_by_hand():
    q, k = np.zeros((2, 1, 4)), np.ones((1, 5, 4))
    lse = np.log(np.full((2, 1), 4.0))
    prev = np.arange(10.0, 15.0)[None]
    # equal scores: a quarter from each row that sees the key
    assert np.allclose(OV.weights(q, lse, k, prev), [[10.5, 11.5, 12.5, 0.5, 0.25]])
    assert np.allclose(OV.weights(q, lse, k, prev, decay=0.5), [[5.5, 6, 6.5, 0.5, 0.25]])
    assert np.allclose(OV.weights(q, lse, k, None, window=2), [[0, 0, 0.25, 0.5, 0.25]])
    lse[1] = np.inf
    assert np.allclose(OV.weights(q, lse, k, None), [[0.25, 0.25, 0.25, 0.25, 0]])
    assert np.allclose(OV.weights(q, lse, k[:, :1], None), [[0]])   # its only row has no lse


@pytest.mark.parametrize("w,keep,sinks,recent,want", [
    ([5, 1, 4, 2, 3], 5, 0, 0, [0, 1, 2, 3, 4]),
    ([5, 1, 4, 2, 3], 9, 3, 3, [0, 1, 2, 3, 4]),
    ([5, 1, 4, 2, 3], 2, 0, 0, [0, 2]),
    ([5, 1, 4, 2, 3], 2, 0, 1, [0, 4]),
    ([5, 1, 4, 2, 3], 3, 2, 0, [0, 1, 2]),
    ([5, 1, 4, 2, 3], 2, 1, 1, [0, 4]),
    ([1, 1, 1, 1, 1], 3, 0, 1, [0, 1, 4]),
    ([0.0, -0.0, 0.0, -1.0, 0.0], 2, 0, 0, [0, 1]),
    ([math.nan, 1, math.nan, -math.inf, 0], 3, 0, 0, [1, 3, 4]),
    ([math.nan, 1, math.nan, math.inf, 0], 4, 0, 0, [0, 1, 3, 4]),
])
def test_kept(w, keep, sinks, recent, want):
    assert OV.kept(np.array(w, dtype=np.float64), keep, sinks, recent) == want


def test_kept_is_the_best_subset():
    r = np.random.default_rng(1)
    for _ in range(50):
        w = r.standard_normal(12)
        got = OV.kept(w, 6, 2, 1)
        assert {0, 1, 11} <= set(got) and len(got) == 6
        out = [j for j in range(12) if j not in got]
        assert min(w[j] for j in got if 2 <= j < 11) > max(w[j] for j in out)
