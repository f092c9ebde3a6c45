"""How far a write of the 8-bit cache can be taken back: the tail holds the
open block and the one before it, so 64 rows always, more where the open block
has rows, and the start of any block."""

import pytest
import torch

from _helpers import DEV, i32_dev, need_gpu
from test_gpu_int8_cache import check, rows
from tree_verify_attention_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("length", [64 * 5, 64 * 5 + 1, 64 * 5 + 40, 64 * 5 + 63])
def test_the_furthest_start(length):
    hkv, d = 2, 64
    k, v = rows(50, length, hkv, d), rows(51, length, hkv, d)
    held = 64 * (length // 64 - 1)               # 64 + length % 64 rows back
    cache = api.Int8Cache(hkv, d, 500, device=DEV)
    cache.append(k.to(DEV), v.to(DEV))
    cache.truncate(held - 1)
    assert int(cache.status) == api.DEV_CTX
    check(cache, k, v, length)
    cache.status.zero_()
    cache.truncate(held + 1)
    cache.append(k[held + 1:].to(DEV), v[held + 1:].to(DEV))
    cache.truncate(held)
    cache.append(k[held:].to(DEV), v[held:].to(DEV))
    assert int(cache.status) == 0
    check(cache, k, v, length)


@pytest.mark.parametrize("back,ok", [(64, True), (65, False)])
def test_a_chain_of_65_nodes_taken_back(back, ok):
    """A chain of 65 accepted rows that ends with a block: 64 of them can go."""
    hkv, d, n = 2, 128, 65
    at = 64 * 6 - n
    k, v = rows(52, at + n, hkv, d), rows(53, at + n, hkv, d)
    cache = api.Int8Cache(hkv, d, 500, device=DEV)
    cache.append(k[:at].to(DEV), v[:at].to(DEV))
    api.kv_commit(cache, i32_dev([n]), i32_dev(list(range(n))), k[at:].to(DEV, torch.bfloat16),
                  v[at:].to(DEV, torch.bfloat16))
    check(cache, k, v, at + n)
    cache.truncate(at + n - back)
    assert int(cache.status) == (0 if ok else api.DEV_CTX)
    check(cache, k, v, at + n - back if ok else at + n)
