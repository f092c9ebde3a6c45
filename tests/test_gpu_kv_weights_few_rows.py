"""Key weights from one or a few query rows of a head (the block-by-block form,
up to 16 rows), at the border to the other form and over many chunks."""

import pytest
import torch

from _helpers import DEV, need_gpu
from tree_verify_attention_gb300 import api
from test_gpu_kv_weights import check, i32, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hkv,hq,n", [(1, 1, 1), (2, 2, 16), (2, 2, 17), (4, 32, 2), (4, 36, 2),
                                      (3, 48, 1), (3, 51, 1), (2, 10, 3)])
def test_rows_about_sixteen(d, hkv, hq, n):
    for C in (n, 100, 1500):
        check(C + hq, hkv, hq, d, max(C, n), "q4_0", n, decay=0.5)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_chunks_of_several_heads(d):
    check(1, 8, 32, d, 40001 // (d // 64), "q4_0", 1)
    check(2, 5, 30, d, 30001 // (d // 64), "q4_0", 2, window=1111)
    check(3, 7, 7, d, 20480 // (d // 64), "q4_0", 16, in_place=True)


def test_magnitudes_of_scales():
    """Cached values up to the end of binary16, and tiny ones."""
    for scale in (300.0, 4000.0, 2.0 ** -10):
        cache, _, _, lse, prev = make(1, 2, 128, 1, 300, "q4_0", 1, 4)
        g = torch.Generator().manual_seed(3)
        k = torch.randn(2, 300, 128, generator=g) * scale
        cache.fill(k.to(DEV), k.to(DEV))
        q = (torch.randn(1, 4, 128, generator=g) / scale).to(torch.bfloat16).to(DEV)
        few, many = torch.empty(2, 300, device=DEV), torch.empty(2, 300, device=DEV)
        api.kv_weights(cache, q, lse, few)
        # the same row again as one of nine, the others without weight
        l9 = torch.full((9, 4), float("inf"), device=DEV)
        l9[8] = lse[0]
        api.kv_weights(cache, q.expand(9, 4, 128).contiguous(), l9, many, status=i32([0]))
        assert torch.isfinite(few).all() and torch.allclose(few, many, rtol=1e-5)
