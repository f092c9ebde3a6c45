"""Query rows of very different size in one tile of the attention over the
8-bit cache: each row's result is its own.

The rows beside an odd one are held to the tolerances of test_gpu_int8_attn.py
for a call without it. They need not be equal to that call's to the bit: the
columns of a softmax group take new references together, whichever of them
asks for it, and a weight's rounding to binary16 goes by its reference."""

import numpy as np
import pytest
import torch

import oracle
from _helpers import need_gpu
from test_gpu_int8_attn import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def expected(c, dtype):
    """The float64 result of a case of ordinary rows, and its tolerances."""
    k, v = c.values()
    q, tk, tv = (t.double().numpy() for t in (c.q, c.tk, c.tv))
    f = oracle.attention.tree_verify_attention_by_head
    want, wlse = f(q, k, v, tk, tv, c.parent, c.ctx, c.window, c.scale)
    mag, _ = f(q, k, np.abs(v), tk, np.abs(tv), c.parent, c.ctx, c.window, c.scale)
    g, qk = c.hq // c.hkv, 0.0
    for h in range(c.hkv):
        keys = np.abs(np.concatenate([k[h], tk[:, h]]))
        qk = max(qk, (np.abs(q[:, h * g:(h + 1) * g].reshape(-1, c.d)) @ keys.T).max())
    delta = (c.d / 16 + 4) * 2.0 ** -22 * qk * c.d ** -0.5
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    tol = mag * (2.0 ** -11 + 2.0 ** -20 + 2 * delta + 2.0 ** -12) + step * np.abs(want) + 1e-30
    return want, tol, wlse, delta + 2.0 ** -20 + 2.0 ** -22 * np.abs(wlse)


def assert_rows(out, lse, ref, rows):
    want, tol, wlse, ltol = ref
    assert (np.abs(out - want)[rows] <= tol[rows]).all()
    assert (np.abs(lse - wlse)[rows] <= ltol[rows]).all()


SHAPES = [(9, 6, 2, 64, 150), (23, 24, 4, 256, 700), (65, 8, 1, 128, 300)]


@pytest.mark.parametrize("n,hq,hkv,d,ctx", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("power", [12, 20, 40, 60, 100, 120])
def test_one_large_row(n, hq, hkv, d, ctx, dtype, power):
    c = Case(n, hq, hkv, d, ctx)
    ref = expected(c, dtype)
    node, head = n // 2, hq - 1
    c.q[node, head] = (c.q[node, head].float() * 2.0 ** power).to(torch.bfloat16)
    out, lse = c.run(dtype)
    rows = np.ones((n, hq), bool)
    rows[node, head] = False
    assert_rows(out, lse, ref, rows)
    # The large row attends to its best key alone: the runner-up is further
    # off than twice a score's error, and than the exponent's range.
    k, v = c.values()
    kv = head // (hq // hkv)
    line, x = [], node
    while x >= 0:
        line.append(x)
        x = int(c.parent[x])
    keys = np.concatenate([k[kv], c.tk.double().numpy()[line, kv]])
    vals = np.concatenate([v[kv], c.tv.double().numpy()[line, kv]])
    q = c.q.double().numpy()[node, head]
    s = keys @ q / d ** 0.5
    delta = (d / 16 + 4) * 2.0 ** -22 * (np.abs(keys) @ np.abs(q)).max() / d ** 0.5
    order = np.argsort(s)[::-1]
    assert s[order[0]] - s[order[1]] > 2 * delta + 40, "the case has no clear best key"
    want = vals[order[0]]
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    assert (np.abs(out[node, head] - want) <= (2.0 ** -11 + step + 2.0 ** -19) * np.abs(want)
            + 2.0 ** -20).all()
    assert abs(lse[node, head] - s.max()) <= delta + 2.0 ** -22 * abs(s.max())


@pytest.mark.parametrize("power", [40, 110])
def test_zero_and_small_rows_beside_a_large_one(power):
    n, hq, hkv, d, ctx = 9, 6, 2, 128, 200
    c = Case(n, hq, hkv, d, ctx)
    c.q[0, 0] = 0.0
    c.q[1, 0] = (c.q[1, 0].float() * 2.0 ** -30).to(torch.bfloat16)
    ref = expected(c, torch.float32)
    c.q[2, 0] = (c.q[2, 0].float() * 2.0 ** power).to(torch.bfloat16)
    out, lse = c.run(torch.float32)
    rows = np.ones((n, hq), bool)
    rows[2, 0] = False
    assert_rows(out, lse, ref, rows)


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("n,hq,hkv,d,ctx,window", [(1, 1, 1, 64, 0, 0), (1, 2, 1, 128, 300, 0),
                                                   (9, 6, 2, 256, 500, 100),
                                                   (65, 12, 2, 64, 900, 0)])
def test_a_row_that_is_not_finite_has_no_result(value, n, hq, hkv, d, ctx, window):
    """Also where every key has the same sign in that place, so that all of
    the row's scores are -inf."""
    def positive(x):
        return torch.cat([x[..., :9], x[..., 9:10].abs() + 1.0, x[..., 10:]], -1)

    def make():
        c = Case(n, hq, hkv, d, ctx, window, k_fun=positive)
        c.tk[..., 9] = c.tk[..., 9].abs() + 1.0
        return c

    good, c = make(), make()
    ref, rlse = good.check(torch.float32)
    c.q[n - 1, hq - 1, 9] = value
    out, lse = c.run(torch.float32)
    rows = np.ones((n, hq), bool)
    rows[n - 1, hq - 1] = False
    assert np.isnan(out[n - 1, hq - 1]).all() and not np.isfinite(lse[n - 1, hq - 1])
    assert np.array_equal(out[rows], ref[rows]) and np.array_equal(lse[rows], rlse[rows])


def test_rows_of_many_sizes_against_the_definition():
    """Every node's rows on a scale of their own, 2^-24 to 2^4."""
    c = Case(30, 4, 1, 128, 400)
    e = torch.linspace(-24, 4, 30).round()[:, None, None]
    c.q = (c.q.float() * torch.exp2(e)).to(torch.bfloat16)
    c.check(torch.float32)
    c.check()


def check_sharp_rows(c, dtype, most_clear):
    """Rows whose best key is ahead of all others by more than a score's error
    (and than the exponent's range) have that key's value; the others, of which
    there are few, a finite one within the values' range."""
    out, lse = c.run(dtype)
    k, v = c.values()
    tk, tv, q = c.tk.double().numpy(), c.tv.double().numpy(), c.q.double().numpy()
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    clear = 0
    for node in range(c.n):
        line, x = [], node
        while x >= 0:
            line.append(x)
            x = int(c.parent[x])
        for head in range(c.hq):
            h = head // (c.hq // c.hkv)
            keys, vals = np.concatenate([k[h], tk[line, h]]), np.concatenate([v[h], tv[line, h]])
            s = keys @ q[node, head] / c.d ** 0.5
            delta = ((c.d / 16 + 4) * 2.0 ** -22
                     * (np.abs(keys) @ np.abs(q[node, head])).max() / c.d ** 0.5)
            best = s.argmax()
            got = out[node, head]
            assert abs(lse[node, head] - s[best]) <= delta + 40 + 2.0 ** -22 * abs(s[best])
            if s[best] - np.delete(s, best).max() > 2 * delta + 40:
                clear += 1
                tol = (2.0 ** -11 + step + 2.0 ** -19) * np.abs(vals[best]) + 2.0 ** -20
                assert (np.abs(got - vals[best]) <= tol).all()
            else:
                assert (np.abs(got) <= np.abs(vals).max() * 1.01).all()
    assert clear >= most_clear * c.n * c.hq


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,hq,hkv,d,ctx", [(1, 4, 2, 64, 900), (23, 12, 2, 256, 700),
                                            (30, 3, 1, 128, 2000)])
@pytest.mark.parametrize("power", [24, 40, 118])
def test_all_rows_large(n, hq, hkv, d, ctx, dtype, power):
    """Scores whose rounding is far above the exponent's range."""
    check_sharp_rows(Case(n, hq, hkv, d, ctx, q_scale=2.0 ** power), dtype, 0.8)


@pytest.mark.parametrize("block", [0, 3, 9])
@pytest.mark.parametrize("power", [21, 30, 36])
def test_a_block_of_large_keys(block, power):
    """Ordinary queries meet them first, last or in between."""
    def large(k):
        k = k.clone()
        k[64 * block:64 * block + 64] *= 2.0 ** power
        return k

    check_sharp_rows(Case(23, 12, 2, 128, 64 * 10 + 9, k_fun=large), torch.float32, 0.8)
    check_sharp_rows(Case(1, 2, 1, 64, 64 * 10 + 9, k_fun=large), torch.bfloat16, 0.5)
