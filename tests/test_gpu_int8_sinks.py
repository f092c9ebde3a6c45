"""One key that takes nearly all of the weight and adds nothing (an attention
sink: a large score, a zero value row): what is left of the output comes from
keys whose weights are about 2^-20 of the largest. Tolerances as in
test_gpu_int8_attn.py, where a weight is rounded to binary16 by 2^-11 of
itself; that has to hold for such weights too."""

import pytest
import torch

from _helpers import need_gpu
from test_gpu_int8_attn import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("n,hq,hkv,d,ctx", [(1, 1, 1, 64, 700), (5, 6, 2, 128, 1000),
                                            (23, 24, 4, 256, 2000), (65, 128, 8, 64, 1500)])
@pytest.mark.parametrize("score", [6.0, 10.0, 14.25])
def test_a_sink_without_a_value(n, hq, hkv, d, ctx, score):
    # the query is 1 in dim 0 (scale 1), the sink's key is `score` there and
    # every other key 0, so all of them weigh e^-score of the sink
    def keys(k):
        k = torch.zeros_like(k)
        k[0, :, 0] = score
        return k

    def values(v):
        v = 1.0 + 0.5 * v.clamp(-1.5, 1.5)
        v[0] = 0.0
        return v

    c = Case(n, hq, hkv, d, ctx, k_fun=keys, v_fun=values, scale=1.0)
    c.q = torch.zeros_like(c.q)
    c.q[..., 0] = 1.0
    c.tk = torch.zeros_like(c.tk)
    c.tv = (1.0 + 0.5 * c.tv.float().clamp(-1.5, 1.5)).to(torch.bfloat16)
    c.check(torch.float32)
    c.check()


@pytest.mark.parametrize("n,hq,hkv,d", [(1, 1, 1, 64), (5, 6, 2, 128), (23, 24, 4, 256)])
@pytest.mark.parametrize("ctx,zeros", [(40, 1), (200, 64), (200, 192)])
@pytest.mark.parametrize("score", [20.0, 44.0, 55.0])
def test_zero_value_rows_and_blocks(n, hq, hkv, d, ctx, zeros, score):
    """The sink in the open block, where rows have scales of their own, and in
    a block (or all of them) without any value: however far its score is ahead
    of the others, there is nothing that their values could be small against."""
    def keys(k):
        k = torch.zeros_like(k)
        k[0, :, 0] = score
        return k

    def values(v):
        v = 1.0 + 0.5 * v.clamp(-1.5, 1.5)
        v[:zeros] = 0.0
        return v

    c = Case(n, hq, hkv, d, ctx, k_fun=keys, v_fun=values, scale=1.0)
    c.q = torch.zeros_like(c.q)
    c.q[..., 0] = 1.0
    c.tk = torch.zeros_like(c.tk)
    c.tv = (1.0 + 0.5 * c.tv.float().clamp(-1.5, 1.5)).to(torch.bfloat16)
    c.check(torch.float32)
    c.check()
