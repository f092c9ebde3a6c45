"""Draws at temperatures near the largest float32, where what lies some 30
temperatures below the largest logit leaves float32: a cut near the end of the
row is the definition's all the same (tolerances as in ``test_gpu_sampling.py``;
no row here lies on a border)."""

import numpy as np
import pytest
import torch

from _helpers import DEV, need_gpu
from test_gpu_sampling import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


# with one CTA a row and with several; the last warp's run full and not
@pytest.mark.parametrize("v", [600, 2000, 2100, 3001, 4900, 20001])
@pytest.mark.parametrize("t", [1e37, 1.2e37, 3e38])
def test_cuts_near_the_end(t, v):
    x, u = make(v, 6, v, torch.float32)
    for f in (dict(top_p=0.95), dict(top_p=0.99), dict(top_k=v - 10),
              dict(top_k=v - 10, top_p=0.95)):
        check(x, u, temperature=t, **f)
        some = torch.cat([x, x.flip(0)]).repeat(8, 1)[:90]     # a CTA a row
        check(some, u.repeat(15), temperature=t, rows=range(0, 90, 11), **f)


@pytest.mark.parametrize("v", [2000, 4900])
def test_top_k_whatever_the_temperature(v):
    """All weights alike: the tokens that stay are the same at any temperature."""
    x, u = make(v + 1, 6, v, torch.float32)
    got = [check(x, u, temperature=t, top_k=v - 10)[0] for t in (1e30, 1e36, 1.2e37, 3e38)]
    assert all(np.array_equal(got[0], g) for g in got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_without_most_tokens(dtype):
    """-inf is below the window, wherever that ends; bf16 and float32."""
    x, u = make(5, 6, 3001, dtype)
    x[:, ::3] = -torch.inf
    for f in (dict(top_p=0.95), dict(top_p=0.99), dict(top_k=1990), dict(top_k=2500)):
        tok, _ = check(x, u, temperature=3e38, few=1, **f)
        assert np.all(tok % 3 != 0)


def test_large_logits_too():
    """Logits of the temperature's size."""
    x, u = make(8, 6, 3001, torch.float32)
    for f in (dict(), dict(top_p=0.95), dict(top_k=2900)):
        check(x * 1e32, u, temperature=1e32, few=1, **f)
