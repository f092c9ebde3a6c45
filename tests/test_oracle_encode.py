"""Pins of the norm-and-rotation oracle: closed forms and invariants, and the
fixed-point turns of ``api.Rope`` against integer arithmetic."""

import math
from fractions import Fraction

import numpy as np
import pytest

import oracle.encode as OE
from tree_verify_attention_gb300 import api


def test_depths():
    assert OE.depths([-1, 0, 1, 1, 3, 0]).tolist() == [0, 1, 2, 2, 3, 1]
    assert OE.depths([7, 5, 1, 3]).tolist() == [0, 1, 2, 1]     # entries outside [0, i) are 0
    assert OE.depths([3]).tolist() == [0]


def test_norm_closed_forms():
    x = np.array([[3.0, 4.0]])
    assert np.allclose(OE.norm(x, None, 0.0), np.array([[3.0, 4.0]]) / math.sqrt(12.5), rtol=1e-15)
    assert np.allclose(OE.norm(x, [2.0, 0.5], 12.5), [[6.0 / 5.0, 2.0 / 5.0]], rtol=1e-15)
    r = np.random.default_rng(0).standard_normal((5, 64))
    assert np.allclose((OE.norm(r, None, 0.0) ** 2).mean(1), 1.0, rtol=1e-14)
    assert np.allclose(OE.norm(1e6 * r, None, 0.0), OE.norm(r, None, 0.0), rtol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation(interleaved):
    f = [math.pi / 2, 0.0]
    y = np.arange(1.0, 7.0).reshape(1, 1, 6)       # the last two dims are not rotated
    got = OE.rotate(y, [1], f, interleaved)[0, 0]
    want = [-2, 1, 3, 4, 5, 6] if interleaved else [-3, 2, 1, 4, 5, 6]
    assert np.allclose(got, want, atol=1e-15)
    # what a query sees of a key depends on the distance alone
    r = np.random.default_rng(1)
    q, k = r.standard_normal((2, 1, 1, 64))
    f = [1e4 ** (-i / 32) for i in range(32)]
    dots = [float((OE.rotate(q, [p + 7], f, interleaved) * OE.rotate(k, [p], f, interleaved)).sum())
            for p in (0, 1, 1000)]
    assert np.allclose(dots, dots[0], rtol=1e-10)


@pytest.mark.parametrize("base,dim", [(1e4, 64), (1e6, 256), (5e5, 128)])
def test_turns(base, dim):
    """Turns per position as 64-bit fractions: within 2^-52 of the frequency
    (relative: a double's division and the reference value of 2 pi)."""
    t = api.Rope(dim, base=base, device="cpu").turns.tolist()
    pi = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    for i, u in enumerate(t):
        u %= 1 << 64
        want = Fraction(base ** (-2.0 * i / dim)) / (2 * pi)
        assert abs(Fraction(u, 1 << 64) - want) <= want / 2 ** 51 + Fraction(1, 1 << 63)
    # frequencies of more than a turn, and negative ones, go by their fraction
    t = api.Rope(64, 16, inv_freq=[2 * math.pi * 1.25, -math.pi / 2] + [0.0] * 6,
                 device="cpu").turns
    assert t[0].item() == 1 << 62 and t[1].item() == -(1 << 62) and not t[2:].any()


def test_rope_refusals():
    for kw in (dict(head_dim=96), dict(head_dim=64, rot_dim=24), dict(head_dim=64, rot_dim=128),
               dict(head_dim=64, rot_dim=-16), dict(head_dim=64, inv_freq=[1.0]),
               dict(head_dim=64, rot_dim=16, inv_freq=[math.inf] * 8),
               dict(head_dim=64, rot_dim=16, inv_freq=[math.nan] * 8)):
        with pytest.raises(api.DfvError):
            api.Rope(device="cpu", **kw)
