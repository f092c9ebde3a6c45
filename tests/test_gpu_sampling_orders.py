"""Draws from rows whose order in the vocabulary misleads counts that are taken
from a part of it: the result is the definition's all the same (tolerances as in
``test_gpu_sampling.py``; of a call's rows one may lie on a border)."""

import pytest
import torch

from _helpers import DEV, need_gpu
from test_gpu_sampling import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def ordered(kind, n, v, g):
    x = torch.randn(n, v, generator=g) * 2
    i = torch.arange(v)
    if kind == "ascending":
        return x.sort(1).values
    if kind == "descending":
        return x.sort(1, descending=True).values
    if kind == "pieces up":          # every eighth piece of 64 tokens far above the others
        return x + 4.0 * ((i // 64) % 8 == 0)
    if kind == "pieces down":
        return x - 4.0 * ((i // 64) % 8 == 0)
    if kind == "halves":
        return x + 5.0 * (i < v // 2)
    if kind == "flat":               # a handful of values, thousands of each
        return torch.round(x / 2) * 0.25
    return x + 3.0 * ((i // 32) % 2 == 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["ascending", "descending", "pieces up", "pieces down", "halves",
                                  "flat", "alternating"])
def test_orders(kind, dtype):
    g = torch.Generator().manual_seed(len(kind))
    for n, v in ((3, 60011), (90, 30007)):
        x = ordered(kind, n, v, g).to(dtype).to(DEV)
        u = torch.rand(n, generator=g).to(DEV)
        for kw in (dict(top_p=0.5), dict(top_p=0.95), dict(top_p=0.99, temperature=1.5),
                   dict(top_k=1000), dict(top_k=5000, top_p=0.9), dict(top_p=0.9, min_p=0.01)):
            check(x, u, rows=range(0, n, 7), few=1, **kw)
