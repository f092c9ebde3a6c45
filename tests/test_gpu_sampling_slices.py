"""Draws from rows around the lengths at which they are cut into more slices, and
the longest ones: a row's draw is the same however it is cut (alone it has up to
sixteen slices), and the definition's (tolerances as in ``test_gpu_sampling.py``;
of a call's checked rows one may lie on a border)."""

import numpy as np
import pytest
import torch

from _helpers import DEV, need_gpu
from test_gpu_sampling import check, make, run
from tree_verify_attention_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


# a slice holds some 38300 bf16 or 19150 float32 tokens
@pytest.mark.parametrize("v", [19152, 38303, 38320, 76639, 76657, 153247, 153264, 153265, 155700,
                               306529, 1 << 19])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_however_it_is_cut(v, dtype):
    one, u1 = make(v, 5, v, dtype, likely=4)
    x, u = one.repeat(16, 1), u1.repeat(16)      # 80 rows: as few slices as hold one
    for f in (dict(), dict(top_p=0.9), dict(top_k=300, top_p=0.95)):
        tok, lp = check(x, u, rows=range(2), few=1, **f)
        alone = run(one[:1], u[:1], api.Sampling(**f))
        few = run(one, u1, api.Sampling(**f))
        assert alone[0][0] == tok[0] and alone[1][0] == lp[0]
        assert np.array_equal(np.tile(few[0], 16), tok) and np.array_equal(np.tile(few[1], 16), lp)
