"""Pins of the sampling oracle: hand-made rows, plain loops, frequencies."""

import itertools
import math

import numpy as np
import pytest

import oracle.sampling as OS

X = [math.log(v) for v in (1.0, 4.0, 2.0, 2.0, 1.0)]       # weights 1 4 2 2 1 of 10


@pytest.mark.parametrize("u,token", [(0.0, 0), (0.0999, 0), (0.1001, 1), (0.4999, 1), (0.5001, 2),
                                     (0.6999, 2), (0.7001, 3), (0.9001, 4), (0.99999, 4)])
def test_index_order(u, token):
    got = OS.draw(X, u)
    assert got[0] == token
    assert math.isclose(got[1], math.log([.1, .4, .2, .2, .1][token]), rel_tol=1e-12)
    assert math.isclose(got[2], min(abs(u - b) for b in (0 if u else 1, .1, .5, .7, .9)),
                        abs_tol=1e-12)


def test_filters_by_hand():
    def ids(**kw):
        k = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
        return OS.kept(X, **{**k, **kw})[0].tolist()

    assert ids() == [0, 1, 2, 3, 4]
    assert ids(top_k=1) == [1] and ids(top_k=2) == [1, 2]       # the tie goes to index 2
    assert ids(top_k=4) == [0, 1, 2, 3]
    assert ids(top_k=5) == ids(top_k=9) == [0, 1, 2, 3, 4]
    assert ids(top_p=0.0) == ids(top_p=0.39) == [1] and ids(top_p=0.41) == [1, 2]
    assert ids(top_p=0.61) == [1, 2, 3] and ids(top_p=0.81) == [0, 1, 2, 3]
    assert ids(min_p=0.24) == [0, 1, 2, 3, 4] and ids(min_p=0.26) == [1, 2, 3]
    assert ids(min_p=0.51) == ids(min_p=1.0) == ids(min_p=7.0) == [1]
    # top-p is a share of what top-k leaves: 6 of 10, half of which is 3 < 4
    assert ids(top_k=2, top_p=0.5) == [1] and ids(top_p=0.5) == [1, 2]
    # temperature 1/2 squares the weights: 1 16 4 4 1 of 26
    assert ids(temperature=0.5, top_p=0.6) == [1] and ids(temperature=0.5, top_p=0.62) == [1, 2]


def test_the_floor_and_rows_without_a_distribution():
    x = [0.0, -27.7, -27.8, -math.inf]
    assert OS.kept(x, 1.0, 0, 1.0, 0.0)[0].tolist() == [0, 1]
    assert OS.draw([math.nan, 1.0], 0.5)[0] == -1 and OS.draw([-math.inf] * 3, 0.5)[0] == -1
    assert OS.draw([math.inf, 1.0], 0.5)[0] == -1
    assert OS.draw([1.0, 3.0, 3.0], 0.9, temperature=0.0)[:2] == (1, 0.0)


def test_frequencies():
    """Evenly spaced random numbers hit each kept token in proportion."""
    r = np.random.default_rng(0)
    x = r.standard_normal(40)
    ids, w, _ = OS.kept(x, 0.7, 20, 0.9, 0.05)
    n = 20000
    got = np.bincount([OS.draw(x, (i + 0.5) / n, 0.7, 20, 0.9, 0.05)[0] for i in range(n)],
                      minlength=40)
    assert np.abs(got[ids] / n - w / w.sum()).max() <= 1.0 / n
    assert got.sum() == got[ids].sum()


def test_walk_against_enumeration():
    for parent in itertools.product(range(1), range(2), range(3)):
        par = (-1,) + parent
        for tokens in itertools.product((5, 6), repeat=3):
            for target in itertools.product((5, 6, -1), repeat=4):
                path, out = OS.walk(par, (0,) + tokens, target)
                for a, b in zip(path, path[1:]):
                    same = [i for i in range(1, 4)
                            if par[i] == a and (0,) + tokens != () and tokens[i - 1] == target[a]]
                    assert b == same[0] and target[a] >= 0
                assert not [i for i in range(1, 4) if par[i] == path[-1] and target[path[-1]] >= 0
                            and tokens[i - 1] == target[path[-1]]]
                assert out == [target[i] for i in path]
