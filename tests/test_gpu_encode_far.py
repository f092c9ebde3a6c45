"""Rotations at far positions against angles of 80 digits: as exact as near ones
(tolerance as in ``test_gpu_encode.py``, whose part for the angle holds the cut
of the turns, 2^31 * 2^-65 of one, as well)."""

import decimal
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from _helpers import DEV, need_gpu
from test_gpu_encode import i32, near_enough, rows
from tree_verify_attention_gb300 import api

pytestmark = pytest.mark.gpu

TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,base", [(256, 256, 1e6), (128, 32, 1e4), (64, 64, 5e5)])
def test_far_positions(d, rot, base, interleaved):
    pos = [0, 131071, (1 << 24) + 1, 123456789, (1 << 30) + 7, (1 << 31) - 1, -(1 << 31)]
    half = rot // 2
    with decimal.localcontext(decimal.Context(prec=60)):
        turns = [Fraction(decimal.Decimal(base) ** (decimal.Decimal(-i) / half)) / TWO_PI
                 for i in range(half)]
    angle = np.array([[2 * math.pi * float(p * t % 1) for t in turns] for p in pos])
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    x = rows(1, len(pos), 3, d, torch.float32)
    out = torch.empty_like(x)
    api.qk_norm_rope(x, None, None, api.Rope(d, rot, base=base, interleaved=interleaved), out, None,
                     eps=None, positions=i32(pos))
    y = x.double().cpu().numpy()
    a = np.arange(half) * 2 if interleaved else np.arange(half)
    b = a + 1 if interleaved else a + half
    want, both = y.copy(), np.abs(y)
    want[..., a], want[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    both[..., a] = both[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    near_enough(out, want, both, torch.float32)
