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


@pytest.mark.parametrize("length,held", [(100, False), (128, True), (230, True), (192, True),
                                         (191, False), (1, False)])
def test_a_length_set_back_directly(length, held):
    """As with the other caches' ctx_len. Inside a block that the tail no
    longer holds the rows of that block are left out, and it is reported."""
    n, hq, hkv, d = 300, 4, 2, 64
    k, v = rows(54, n, hkv, d, spread=False), rows(55, n, hkv, d, spread=False)
    cache, short = (api.Int8Cache(hkv, d, 400, device=DEV) for _ in range(2))
    cache.append(k.to(DEV), v.to(DEV))          # holds blocks 3 and 4
    cache.ctx_len.fill_(length)
    seen = length if held else length // 64 * 64
    short.append(k[:seen].to(DEV), v[:seen].to(DEV))
    g = torch.Generator(device=DEV).manual_seed(8)
    q, tk, tv = (torch.randn(3, h, d, generator=g, device=DEV).to(torch.bfloat16)
                 for h in (hq, hkv, hkv))
    ws = api.workspace(api.int8_attn_workspace_bytes(3, hq, hkv, d, 0, 400))
    outs = []
    for c in (cache, short):
        out, lse = torch.empty(3, hq, d, device=DEV), torch.empty(3, hq, device=DEV)
        api.tree_verify_attn(c, q, tk, tv, i32_dev([-1, 0, 0]), 0, 3, out, lse, ws)
        outs.append((out, lse))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert int(cache.status) == (0 if held else api.DEV_CTX)
    cache.status.zero_()
    got = [torch.full((length, hkv, d), 7.0, device=DEV) for _ in range(2)]
    want = [torch.full((length, hkv, d), 7.0, device=DEV) for _ in range(2)]
    cache.read(0, length, *got)
    short.read(0, seen, want[0][:seen], want[1][:seen])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert int(cache.status) == (0 if held else api.DEV_CTX)
