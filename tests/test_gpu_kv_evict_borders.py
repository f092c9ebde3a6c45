"""Selections where the smallest kept weight is a NaN, an infinity, a zero of
either sign, one of many equal ones or a pinned position's, in caches of one and
of several CTAs a head and of more positions than these hold (equal to the plain
selection of ``oracle/eviction.py``)."""

import math

import pytest
import torch

from _helpers import DEV, need_gpu
from test_gpu_kv_evict import check, filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def weights_of(kind, hkv, cap, g):
    w = torch.rand(hkv, cap, generator=g)
    few = torch.rand(hkv, cap, generator=g)
    if kind == "nan":
        w[:] = math.nan
    elif kind == "mostly nan":
        w[few < 0.9] = math.nan
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "infinities":
        w[few < 0.6] = math.inf
        w[few > 0.7] = -math.inf
    elif kind == "zeros":
        w[:] = 0.0
        w[few < 0.5] = -0.0
        w[few > 0.9] = 1e-45
    elif kind == "two values":
        w = torch.where(few < 0.5, torch.nextafter(torch.tensor(0.5), torch.tensor(1.0)), 0.5)
    elif kind == "all signs":
        w = torch.exp(30 * (few - 0.5)) * torch.sign(w - 0.5)
    return w.to(DEV)


@pytest.mark.parametrize("kind", ["nan", "mostly nan", "equal", "infinities", "zeros",
                                  "two values", "all signs"])
@pytest.mark.parametrize("hkv,C,cap", [(1, 1, 1), (3, 33, 40), (2, 2049, 5000), (5, 9000, 9000),
                                       (1, 40003, 300_000)])
def test_borders(kind, hkv, C, cap):
    g = torch.Generator().manual_seed(C)
    cache, _ = filled(C, hkv, 64, C, cap, "q4_0")
    w = weights_of(kind, hkv, cap, g)
    for keep in sorted({1, max(1, C // 3), max(1, C - 1), C}):
        check(cache, w, keep)
        check(cache, w, keep, sinks=keep)
        check(cache, w, keep, recent=keep)
        check(cache, w, keep, sinks=keep // 2, recent=keep - keep // 2)
        check(cache, w, keep, sinks=keep // 3, recent=keep // 4)


def test_an_empty_cache():
    cache, w = filled(3, 2, 64, 0, 500, "f16")
    check(cache, w, 7, sinks=2, recent=5)
