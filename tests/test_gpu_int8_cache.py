"""The 8-bit cache on the GPU: appending, committing, rolling back and reading
back, bit for bit against the definition in ``oracle/int8.py`` (codes and
scales have one right value, so nothing here has a tolerance)."""

import ctypes

import numpy as np
import pytest
import torch

import oracle.int8 as I8
from _helpers import DEV, need_gpu
from tree_verify_attention_gb300 import _lib, api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def rows(seed, n, hkv, d, spread=True):
    """bf16-valued float32 rows [n, hkv, d] with magnitudes over a wide range."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, hkv, d, generator=g)
    if spread:
        x = x * torch.exp2(torch.randint(-12, 13, (n, hkv, d), generator=g).float())
    return x.to(torch.bfloat16).float()


def check(cache, k, v, n):
    """Content of ``cache`` after the rows k, v [n, hkv, d] were committed."""
    assert int(cache.ctx_len) == n
    nb = n // 64
    for rws, codes, scale, tail, unpack in ((k, cache.k, cache.k_scale, cache.k_tail, I8.unpack_k),
                                            (v, cache.v, cache.v_scale, cache.v_tail, I8.unpack_v)):
        r = rws[:n].permute(1, 0, 2).numpy()
        want_c, want_s = I8.encode_blocks(r)
        assert np.array_equal(unpack(codes.cpu().numpy())[:, :nb], want_c)
        assert np.array_equal(scale.cpu().numpy()[:, :nb], want_s)
        assert np.array_equal(tail.float().cpu().numpy()[:, nb % 2, :n % 64], r[:, nb * 64:])


def read(cache, pos, n, dtype):
    k = torch.full((n, cache.n_kv_heads, cache.head_dim), 7.0, dtype=dtype, device=DEV)
    v = k.clone()
    cache.read(pos, n, k, v)
    return k, v


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pieces", [[1], [63], [64], [65], [300], [1, 62, 1, 1, 63, 64, 65, 128, 7],
                                    [40, 200], [100, 1, 191]])
def test_append_in_pieces(d, dtype, pieces):
    n, hkv = sum(pieces), 3
    k, v = rows(1, n, hkv, d), rows(2, n, hkv, d)
    cache = api.Int8Cache(hkv, d, n + 5, device=DEV)
    at = 0
    for c in pieces:
        cache.append(k[at:at + c].to(DEV, dtype), v[at:at + c].to(DEV, dtype))
        at += c
    assert int(cache.status) == 0 and cache.state[1].item() == 0
    check(cache, k, v, n)
    want_k = I8.cached_values(k.permute(1, 0, 2).numpy()).transpose(1, 0, 2)
    want_v = I8.cached_values(v.permute(1, 0, 2).numpy()).transpose(1, 0, 2)
    for pos, m in ((0, n), (n // 3, n - n // 3), (n - 1, 1)):
        gk, gv = read(cache, pos, m, torch.float32)
        # code * scale rounded once to float32
        assert np.array_equal(gk.cpu().numpy(), want_k[pos:pos + m].astype(np.float32))
        assert np.array_equal(gv.cpu().numpy(), want_v[pos:pos + m].astype(np.float32))
        bk, bv = read(cache, pos, m, torch.bfloat16)
        assert torch.equal(bk, gk.to(torch.bfloat16)) and torch.equal(bv, gv.to(torch.bfloat16))


@pytest.mark.parametrize("hkv,d,n,at", [(8, 256, 64 * 60, 0), (8, 256, 64 * 60 + 17, 45),
                                        (16, 128, 64 * 90 + 63, 64), (32, 64, 64 * 85 + 1, 127),
                                        (3, 256, 64 * 250 + 31, 5)])
def test_long_writes(hkv, d, n, at):
    """Long bf16 writes take their inner blocks through another kernel."""
    k, v = rows(35, at + n, hkv, d), rows(36, at + n, hkv, d)
    v[at + 300, hkv - 1, 3] = float("inf")
    kd, vd = k.to(DEV, torch.bfloat16), v.to(DEV, torch.bfloat16)
    v[at + 300, hkv - 1, 3] = 0.0
    cache = api.Int8Cache(hkv, d, at + n + 10, device=DEV)
    cache.append(kd[:at], vd[:at])
    cache.append(kd[at:], vd[at:])
    assert int(cache.status) == api.DEV_NONFINITE
    check(cache, k, v, at + n)
    if at:      # the same place again, refused: its block is no longer held
        before = cache.k.clone()
        cache.status.zero_()
        cache.append(vd[at:], kd[at:], at=at if at % 64 else at + 1)
        assert int(cache.status) == api.DEV_CTX and torch.equal(cache.k, before)
    cache.append(vd, kd, at=0)
    check(cache, v, k, at + n)
    other = api.Int8Cache(hkv, d, at + n + 10, device=DEV)
    other.append(k.to(DEV), v.to(DEV))        # float32 rows take the other path
    check(other, k, v, at + n)


def test_float_rows_are_rounded_to_bf16_first():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(130, 2, 64, generator=g)
    cache = api.Int8Cache(2, 64, 130, device=DEV)
    cache.append(x.to(DEV), x.to(DEV))
    b = x.to(torch.bfloat16).float()
    check(cache, b, b, 130)


def test_ties_round_to_even():
    """127 x / amax is a half-way point for x = amax / 2 (63.5), and for odd
    x with amax = 254."""
    x = torch.zeros(64, 1, 64)
    x[0, 0, 0] = 254.0
    x[1, 0, :50] = torch.arange(-25, 25).float() * 2 + 1
    y = torch.full((64, 1, 64), 1.0)
    for i in range(64):
        y[i] = 1.0 + i / 128
    y[5, 0] = y.amax() / 2
    cache = api.Int8Cache(1, 64, 64, device=DEV)
    cache.append(x.to(DEV), y.to(torch.bfloat16).float().to(DEV))
    check(cache, x, y.to(torch.bfloat16).float(), 64)


@pytest.mark.parametrize("layout", ["head_major", "padded", "odd_base", "odd_stride",
                                    "reversed_k_v"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides(layout, dtype):
    n, hkv, d = 150, 4, 128
    k, v = rows(4, n, hkv, d), rows(5, n, hkv, d)
    cache = api.Int8Cache(hkv, d, n, device=DEV)
    kd, vd = k.to(DEV, dtype), v.to(DEV, dtype)
    head_major = False
    if layout == "head_major":
        kd, vd, head_major = kd.transpose(0, 1).contiguous(), vd.transpose(0, 1).contiguous(), True
    elif layout == "padded":
        both = torch.empty(n, hkv, 2 * d, dtype=dtype, device=DEV)   # K and V of one projection
        both[..., :d], both[..., d:] = kd, vd
        kd, vd = both[..., :d], both[..., d:]
    elif layout == "odd_base":
        buf = torch.empty(2, n * hkv * d + 1, dtype=dtype, device=DEV)
        buf[0, 1:], buf[1, 1:] = kd.reshape(-1), vd.reshape(-1)
        kd, vd = buf[0, 1:].view(n, hkv, d), buf[1, 1:].view(n, hkv, d)
    elif layout == "odd_stride":
        buf = torch.zeros(2, n, hkv * d + 3, dtype=dtype, device=DEV)
        buf[0, :, :hkv * d], buf[1, :, :hkv * d] = kd.reshape(n, -1), vd.reshape(n, -1)
        kd, vd = (buf[i, :, :hkv * d].unflatten(1, (hkv, d)) for i in range(2))
    else:
        kd = kd.transpose(0, 1).contiguous().transpose(0, 1)   # differs from V's strides
    cache.append(kd, vd, head_major=head_major)
    check(cache, k, v, n)
    # and out, into the same kinds of views
    want, _ = read(cache, 0, n, torch.float32)
    big = torch.full((hkv, n, 2 * d + 1), 3.0, device=DEV)
    out_k, out_v = big[..., :d].transpose(0, 1), big[..., d:2 * d].transpose(0, 1)
    cache.read(0, n, out_k, out_v)
    assert torch.equal(out_k, want) and bool((big[..., -1] == 3.0).all())
    cache.read(0, n, out_k.transpose(0, 1), out_v.transpose(0, 1), head_major=True)
    assert torch.equal(out_k, want)


@pytest.mark.parametrize("back", [1, 5, 40, 64, 100])
def test_rollback_within_the_held_blocks(back):
    """From 64 m + 40 rows, up to 104 can be taken back."""
    n, hkv, d = 64 * 3 + 40, 2, 128
    k, v = rows(6, n, hkv, d), rows(7, n, hkv, d)
    k2, v2 = rows(8, 150, hkv, d), rows(9, 150, hkv, d)
    cache = api.Int8Cache(hkv, d, 400, device=DEV)
    cache.append(k.to(DEV), v.to(DEV))
    cache.truncate(n - back)
    check(cache, k, v, n - back)
    cache.append(k2.to(DEV), v2.to(DEV))
    assert int(cache.status) == 0
    check(cache, torch.cat([k[:n - back], k2]), torch.cat([v[:n - back], v2]), n - back + 150)


def test_rollback_beyond_the_held_blocks_is_refused():
    n, hkv, d = 64 * 4 + 10, 1, 64
    k, v = rows(10, n, hkv, d), rows(11, n, hkv, d)
    cache = api.Int8Cache(hkv, d, 400, device=DEV)
    cache.append(k.to(DEV), v.to(DEV))
    cache.truncate(64 * 3 + 5)          # block 3 is open again, block 2's rows are gone
    assert int(cache.status) == 0
    cache.truncate(64 * 2 + 60)
    assert int(cache.status) == api.DEV_CTX
    check(cache, k, v, 64 * 3 + 5)
    cache.status.zero_()
    cache.truncate(64 * 2)              # a block's start needs no rows
    check(cache, k, v, 64 * 2)
    cache.truncate(64 * 2 + 1)          # nothing lies there any more
    assert int(cache.status) == api.DEV_CTX
    cache.status.zero_()
    cache.append(k[:70].to(DEV), v[:70].to(DEV), at=0)
    check(cache, k, v, 70)
    cache.truncate(5)
    assert int(cache.status) == 0
    check(cache, k, v, 5)


def test_repeated_write_at_one_place():
    """A write at a fixed position gives the same content each time."""
    n, hkv, d, at = 100, 2, 64, 90
    k, v = rows(12, at + n, hkv, d), rows(13, at + n, hkv, d)
    cache = api.Int8Cache(hkv, d, 256, device=DEV)
    cache.append(k[:at].to(DEV), v[:at].to(DEV))
    k2, v2 = k[at:at + 20].to(DEV), v[at:at + 20].to(DEV)
    for _ in range(3):
        cache.append(k2, v2, at=at)
        check(cache, k, v, at + 20)
    assert int(cache.status) == 0


def test_capacity_and_length_errors_write_nothing():
    hkv, d = 2, 64
    k, v = rows(14, 200, hkv, d), rows(15, 200, hkv, d)
    cache = api.Int8Cache(hkv, d, 130, device=DEV)
    cache.append(k[:100].to(DEV), v[:100].to(DEV))
    before = [t.clone() for t in (cache.k, cache.v, cache.k_tail, cache.v_tail, cache.state)]
    cache.append(k[:31].to(DEV), v[:31].to(DEV))               # 131 > 130: the device sees it
    assert int(cache.status) == api.DEV_CAPACITY
    cache.status.zero_()
    cache.append(k[:3].to(DEV), v[:3].to(DEV), at=101)         # a gap
    assert int(cache.status) == api.DEV_CTX
    for a, b in zip(before, (cache.k, cache.v, cache.k_tail, cache.v_tail, cache.state)):
        assert torch.equal(a, b)
    cache.append(k[100:130].to(DEV), v[100:130].to(DEV))
    check(cache, k, v, 130)
    cache.ctx_len.fill_(131)
    cache.status.zero_()
    cache.append(k[:1].to(DEV), v[:1].to(DEV))
    assert int(cache.status) == api.DEV_CTX


@pytest.mark.parametrize("dtype", [0, 1])
def test_a_write_whose_end_passes_31_bits(dtype):
    # The largest capacity, full, and as many rows again: refused on the
    # device before anything but the state is read, so small buffers do.
    cap = 1 << 30
    buf = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    state = torch.tensor([cap, 0, cap // 64 - 1, 0], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    a = buf.data_ptr()
    c = _lib.Kv8CacheStruct(1, 64, cap, 0, state.data_ptr(), a, a, a, a, a, a)
    st = torch.cuda.current_stream().cuda_stream
    assert _lib.load().dfv_kv8_append(ctypes.addressof(c), -1, cap, a, a, dtype, 0, 0, 0, 0,
                                      status.data_ptr(), st) == 0
    torch.cuda.synchronize()
    assert int(status) == api.DEV_CAPACITY
    assert state.tolist() == [cap, 0, cap // 64 - 1, 0] and not buf.any()


def test_untouched_blocks_stay_as_they_are():
    hkv, d = 2, 128
    k, v = rows(16, 70, hkv, d), rows(17, 70, hkv, d)
    cache = api.Int8Cache(hkv, d, 300, device=DEV)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        t.fill_(77)
    cache.append(k.to(DEV), v.to(DEV))
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        assert bool((t[:, 1:] == 77).all())
    check(cache, k, v, 70)


def test_reading_behind_the_committed_rows():
    hkv, d = 2, 64
    k, v = rows(18, 100, hkv, d), rows(19, 100, hkv, d)
    cache = api.Int8Cache(hkv, d, 300, device=DEV)
    cache.append(k.to(DEV), v.to(DEV))
    gk, gv = read(cache, 90, 40, torch.bfloat16)
    assert int(cache.status) == api.DEV_CTX
    assert torch.equal(gk[:10].float().cpu(), k[90:]) and bool((gk[10:] == 7).all())
    assert torch.equal(gv[:10].float().cpu(), v[90:]) and bool((gv[10:] == 7).all())


def test_values_that_are_not_stored():
    hkv, d, n = 2, 64, 130
    k, v = rows(20, n, hkv, d), rows(21, n, hkv, d)
    kd, vd = k.clone(), v.clone()
    kd[3, 0, 5], kd[70, 1, 6], kd[129, 0, 7] = float("nan"), float("inf"), -float("inf")
    vd[0, 0, 0], vd[128, 1, 1] = 2.0 ** 40, -3e38
    for a, b in ((k, kd), (v, vd)):
        a[~torch.isfinite(b) | (b.abs() >= 2.0 ** 40)] = 0.0
    for dtype in (torch.float32, torch.bfloat16):
        cache = api.Int8Cache(hkv, d, n, device=DEV)
        cache.append(kd.to(DEV, dtype), vd.to(DEV, dtype))
        assert int(cache.status) == api.DEV_NONFINITE
        check(cache, k, v, n)


def test_tiny_and_zero_blocks():
    hkv, d = 1, 64
    k = torch.zeros(192, hkv, d)
    k[64:128] = 2.0 ** -41
    k[130] = 2.0 ** -39
    v = rows(22, 192, hkv, d) * 2.0 ** -30
    cache = api.Int8Cache(hkv, d, 192, device=DEV)
    cache.append(k.to(DEV), v.to(DEV))
    check(cache, k, v, 192)
    assert cache.k_scale[0, :2].tolist() == [0.0, 0.0] and float(cache.k_scale[0, 2]) > 0


@pytest.mark.parametrize("ctx", [0, 1, 60, 63, 64, 200])
@pytest.mark.parametrize("n,length", [(1, 1), (23, 1), (23, 9), (65, 65)])
def test_commit(ctx, n, length):
    hkv, d = 4, 256
    k, v = rows(23, ctx, hkv, d), rows(24, ctx, hkv, d)
    tk, tv = rows(25, n, hkv, d), rows(26, n, hkv, d)
    rng = np.random.default_rng(ctx + n)
    path = np.sort(rng.choice(n, length, replace=False)).astype(np.int32)
    cache = api.Int8Cache(hkv, d, 300, device=DEV)
    cache.append(k.to(DEV), v.to(DEV))
    full = torch.full((n,), -1, dtype=torch.int32)
    full[:length] = torch.from_numpy(path)
    L = torch.tensor([length], dtype=torch.int32, device=DEV)
    api.kv_commit(cache, L, full.to(DEV), tk.to(DEV, torch.bfloat16), tv.to(DEV, torch.bfloat16))
    assert int(cache.status) == 0
    check(cache, torch.cat([k, tk[path]]), torch.cat([v, tv[path]]), ctx + length)


def test_commit_the_same_node_twice_and_bad_paths():
    hkv, d, n = 2, 64, 5
    tk, tv = rows(27, n, hkv, d), rows(28, n, hkv, d)
    args = tk.to(DEV, torch.bfloat16), tv.to(DEV, torch.bfloat16)

    def dev(*x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    cache = api.Int8Cache(hkv, d, 10, device=DEV)
    api.kv_commit(cache, dev(3), dev(0, 2, 2, -1, -1), *args)
    assert int(cache.status) == 0
    i = [0, 2, 2]
    check(cache, tk[i], tv[i], 3)
    for L, path in ((2, (0, 5, 0, 0, 0)), (2, (0, -1, 0, 0, 0)), (0, (0, 0, 0, 0, 0)),
                    (6, (0, 0, 0, 0, 0))):
        cache.status.zero_()
        api.kv_commit(cache, dev(L), dev(*path), *args)
        assert int(cache.status) == api.DEV_BAD_PATH
        check(cache, tk[i], tv[i], 3)
    cache.status.zero_()
    api.kv_commit(cache, dev(5), dev(0, 1, 2, 3, 4), *args)
    api.kv_commit(cache, dev(5), dev(0, 1, 2, 3, 4), *args)    # 13 > 10
    assert int(cache.status) == api.DEV_CAPACITY and int(cache.ctx_len) == 8


def test_captured_appends_replay():
    """A captured append advances the length it finds on the device."""
    hkv, d, n = 2, 128, 30
    k, v = rows(29, n, hkv, d), rows(30, n, hkv, d)
    kd, vd = k.to(DEV), v.to(DEV)
    cache = api.Int8Cache(hkv, d, 200, device=DEV)
    cache.append(kd, vd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append(kd, vd)
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    check(cache, k.repeat(5, 1, 1), v.repeat(5, 1, 1), 150)


def test_another_stream():
    hkv, d, n = 2, 128, 200
    k, v = rows(31, n, hkv, d), rows(32, n, hkv, d)
    kd, vd = k.to(DEV), v.to(DEV)
    cache = api.Int8Cache(hkv, d, n, device=DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    cache.append(kd[:77], vd[:77], stream=side)
    with torch.cuda.stream(side):
        cache.append(kd[77:], vd[77:])
    side.synchronize()
    check(cache, k, v, n)


def test_offsets_past_31_bits():
    """Eight heads of 256 at a capacity of 1.2 million: the last head's codes
    start 2.1 GB into the buffer."""
    hkv, d, n = 8, 256, 130
    k, v = rows(33, n, hkv, d), rows(34, n, hkv, d)
    cache = api.Int8Cache(hkv, d, 1_200_000, device=DEV)
    cache.append(k.to(DEV), v.to(DEV))
    gk, gv = read(cache, 0, n, torch.float32)
    for got, r in ((gk, k), (gv, v)):
        want = I8.cached_values(r.permute(1, 0, 2).numpy()).transpose(1, 0, 2)
        assert np.array_equal(got.cpu().numpy(), want.astype(np.float32))
