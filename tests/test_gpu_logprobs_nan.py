"""Rows of logits that hold a NaN: no result of such a row is a number,
wherever the NaN lies, and the rows beside it keep theirs.

Tolerance of the rows beside it: a term exp(z) is within 2^-20 relative where
it counts (ex2.approx 2^-22, the rounding of its argument 2^-24 |z log2 e|). A
thread adds 16 or 32 values of a chunk as pairs, then one sum per chunk, and
lanes, warps and CTAs join in at most 20 more additions: below 64 additions of
2^-24 for the sizes here. So log s is within 2^-20 + 2^-18; differences with it
round to 2^-24 of their size, twice."""

import numpy as np
import pytest
import torch

import oracle.logprobs as OL
from _helpers import DEV, need_gpu
from tree_verify_attention_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


NAN, INF = float("nan"), float("inf")


def poison(kind, x):
    """A row of logits with NaN in it."""
    v = x.numel()
    if kind == "first_half":             # a failed shard of the vocabulary
        x[:v // 2] = NAN
    elif kind == "last_half":
        x[v // 2:] = NAN
    elif kind == "one_among_masked":     # +inf logits under a mask of -inf
        x[v // 4:] = -INF
        x[v * 3 // 4] = NAN
    elif kind == "masked_head":          # what is finite comes after the NaN
        x[:v - v // 4] = -INF
        x[v // 3] = NAN
    elif kind == "four":
        x[v // 2:v // 2 + 4] = NAN
    elif kind == "negative_nan":
        x[:] = -INF
        x[0] = 1.0
        x[v - 1] = torch.tensor([-1], dtype=torch.int32).view(torch.float32)[0]
    elif kind == "all":
        x[:] = NAN


KINDS = ["first_half", "last_half", "one_among_masked", "masked_head", "four", "negative_nan",
         "all"]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v", [(1, 33), (1, 1000), (5, 4000), (1, 151936), (23, 151936),
                                 (70, 1000), (700, 5003), (320, 40009)])
@pytest.mark.parametrize("kind", KINDS)
def test_nan_anywhere_in_a_row(kind, n, v, dtype):
    g = torch.Generator().manual_seed(n + v)
    x = torch.randn(n, v, generator=g) * 2.5
    t = torch.randint(0, v, (n,), generator=g)
    bad = list(range(0, n, 3))
    for r in bad:
        poison(kind, x[r])
    x = x.to(dtype)
    top = min(8, v)
    lp, ent = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    ids = torch.full((n, top), -9, dtype=torch.int32, device=DEV)
    tlp = torch.zeros(n, top, device=DEV)
    api.token_logprobs(x.to(DEV), t.to(DEV, torch.int32), lp, ent, ids, tlp)
    lp, ent, ids, tlp = (o.cpu().numpy() for o in (lp, ent, ids, tlp))
    assert np.isnan(lp[bad]).all() and np.isnan(ent[bad]).all() and np.isnan(tlp[bad]).all()
    assert ((0 <= ids) & (ids < v)).all()
    good = [r for r in range(n) if r % 3]
    if good:
        xs = x[good].float().numpy().astype(np.float64)
        want = OL.token_logprobs(xs, t[good].numpy(), top)
        tol = 2.0 ** -20 + 2.0 ** -18
        assert np.array_equal(ids[good], want[2])
        assert (np.abs(lp[good] - want[0]) <= tol + 2.0 ** -22 * np.abs(want[0])).all()
        assert (np.abs(tlp[good] - want[3]) <= tol + 2.0 ** -22 * np.abs(want[3])).all()
    # and without alternatives (which may split the rows otherwise)
    lp2, ent2 = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    api.token_logprobs(x.to(DEV), t.to(DEV, torch.int32), lp2, ent2)
    lp2, ent2 = lp2.cpu().numpy(), ent2.cpu().numpy()
    assert np.isnan(lp2[bad]).all() and np.isnan(ent2[bad]).all()
    if good:
        assert (np.abs(lp2[good] - want[0]) <= tol + 2.0 ** -22 * np.abs(want[0])).all()
        assert np.isfinite(ent2[good]).all()
