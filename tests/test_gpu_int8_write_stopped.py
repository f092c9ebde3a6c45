"""What a write of the 8-bit cache does after a bounded wait of a long write has
given up: the cache's word for it is set from the host here. Nothing is
written and the length stays, until the word is cleared."""

import pytest
import torch

from _helpers import DEV, i32_dev, need_gpu
from test_gpu_int8_cache import check, rows
from tree_verify_attention_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("call", ["append", "append_at", "long", "long_at", "f32", "commit",
                                  "truncate"])
def test_a_stopped_cache_refuses_writes(call):
    hkv, d, n = 8, 256, 64 * 60 + 17
    k, v = rows(40, n, hkv, d), rows(41, n, hkv, d)
    kd, vd = k.to(DEV, torch.bfloat16), v.to(DEV, torch.bfloat16)
    cache = api.Int8Cache(hkv, d, 2 * n, device=DEV)
    cache.append(kd[:150], vd[:150])
    run, after = {
        "append": (lambda: cache.append(kd[150:160], vd[150:160]), 160),
        "append_at": (lambda: cache.append(kd[140:160], vd[140:160], at=140), 160),
        "long": (lambda: cache.append(kd[150:], vd[150:]), n),
        "long_at": (lambda: cache.append(kd, vd, at=0), n),
        "f32": (lambda: cache.append(kd[150:].float(), vd[150:].float()), n),
        "commit": (lambda: api.kv_commit(cache, i32_dev([3]), i32_dev([0, 1, 2, 3]),
                                         kd[150:154].contiguous(), vd[150:154].contiguous()), 153),
        "truncate": (lambda: cache.truncate(140), 140),
    }[call]
    cache.state[3] = 1
    parts = (cache.k, cache.v, cache.k_scale, cache.v_scale, cache.open_end)
    before = [t.clone() for t in parts]
    for _ in range(2):
        run()
    assert int(cache.status) == api.DEV_TIMEOUT
    for a, b in zip(before, parts):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    cache.state[3] = 0
    cache.status.zero_()
    run()
    assert int(cache.status) == 0
    check(cache, k, v, after)
