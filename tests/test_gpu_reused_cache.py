"""A cache that an eviction wrote to, filled again for the next sequence."""

import numpy as np
import pytest
import torch

from _helpers import DEV, need_gpu
from test_gpu_encode import near_enough, want_of
from tree_verify_attention_gb300 import api

pytestmark = pytest.mark.gpu

HKV, D, CAP, KEEP = 2, 64, 120, 50


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def rows(seed, n):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(HKV, n, D, generator=g).to(DEV) for _ in range(2)]


def evicted(fmt, n=100):
    """A cache of KEEP rows that eviction left of n."""
    full, into = (api.KVCache(HKV, D, CAP, fmt=fmt) for _ in range(2))
    full.fill(*rows(1, n))
    weights = torch.rand(HKV, CAP, generator=torch.Generator().manual_seed(2)).to(DEV)
    api.kv_evict(full, weights, into, torch.empty(HKV, KEEP, dtype=torch.int32, device=DEV))
    assert int(into.ctx_len) == KEEP and int(into.dropped) == n - KEEP
    return into


@pytest.mark.parametrize("fmt", ["q4_0", "f16"])
def test_another_sequence(fmt):
    cache = evicted(fmt)
    cache.fill(*rows(3, 30))
    assert int(cache.ctx_len) == 30 and int(cache.dropped) == 0
    # what comes next stands where the new sequence goes on
    n, hq = 5, 4
    x = torch.randn(n, hq, D, generator=torch.Generator().manual_seed(4)).to(DEV)
    out = torch.empty_like(x)
    api.qk_norm_rope(x, None, None, api.Rope(D), out, None, ctx_len=cache.ctx_len,
                     dropped=cache.dropped)
    freq = [1e4 ** (-2.0 * i / D) for i in range(D // 2)]
    near_enough(out, *want_of(x, None, 1e-6, 30 + np.arange(n), freq, False), torch.float32)
    # and an eviction counts its own rows alone
    into = api.KVCache(HKV, D, CAP, fmt=fmt)
    into.dropped.fill_(77)
    kept = torch.empty(HKV, 20, dtype=torch.int32, device=DEV)
    api.kv_evict(cache, torch.rand(HKV, CAP, device=DEV), into, kept)
    assert int(into.ctx_len) == 20 and int(into.dropped) == 10


def test_rows_behind_the_ones_that_stayed():
    """A fill that goes on with the sequence leaves the count as it is."""
    cache = evicted("f16")
    cache.fill(*rows(5, 20), pos0=KEEP)
    assert int(cache.ctx_len) == KEEP + 20 and int(cache.dropped) == 50
    cache.fill(*rows(6, 1))
    assert int(cache.ctx_len) == 1 and int(cache.dropped) == 0


def test_on_another_stream():
    """The length and the count follow the rows on the stream that was given,
    whatever the current one is at."""
    cache, side = evicted("q4_0"), torch.cuda.Stream()
    k, v = rows(7, 40)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)        # some 50 ms of the current stream
    cache.fill(k, v, stream=side)
    with torch.cuda.stream(side):
        got = torch.cat([cache.ctx_len, cache.dropped])
    side.synchronize()
    assert got.tolist() == [40, 0]
    torch.cuda.synchronize()
    assert int(cache.ctx_len) == 40 and int(cache.dropped) == 0
