"""Log probabilities, entropy and top alternatives on the GPU against the
float64 definition (``oracle/logprobs.py``).

Tolerances. ex2.approx is within 2^-22 relative and the exponent's rounding
adds 2^-24 |z log2 e|, |z| <= 90 where it still counts (below, exp(z) is under
the smallest normal number): a term of the sum is off by at most 2^-22 + 130 *
2^-24 = 2^-16.6 relative in the far tail and 2^-21 for |z| < 4; the sum, whose
terms weigh by their size, stays below 2^-20, and adding v values in 256
threads adds (v / 256 + 20) 2^-24. log s is off by that, and x - m and log s
round to 2^-24 of their size."""

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


def run(logits, tokens, top):
    n = logits.shape[0]
    lp = torch.full((n,), 9.0, device=DEV)
    ent = torch.full((n,), 9.0, device=DEV)
    ids = torch.full((n, top), -9, dtype=torch.int32, device=DEV)
    tlp = torch.full((n, top), 9.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    api.token_logprobs(logits, tokens.to(DEV, torch.int32), lp, ent, ids, tlp, status=st)
    return lp.cpu().numpy(), ent.cpu().numpy(), ids.cpu().numpy(), tlp.cpu().numpy(), int(st)


def check(logits, tokens, top):
    lp, ent, ids, tlp, st = run(logits, tokens, top)
    x = logits.float().cpu().numpy().astype(np.float64)
    want = OL.token_logprobs(x, tokens.numpy(), top)
    v = x.shape[1]
    base = 2.0 ** -20 + (v / 256 + 20) * 2.0 ** -24
    assert st == 0
    assert np.array_equal(ids, want[2])

    def near(got, ref, extra=0.0):
        fin = np.isfinite(ref)
        assert np.array_equal(got[~fin], ref[~fin])
        tol = base + extra + 2.0 ** -22 * np.abs(ref[fin]) + 1e-7
        assert np.all(np.abs(got[fin] - ref[fin]) <= tol)

    near(lp, want[0])
    near(tlp, want[3])
    # each term p z errs like its p (|z| of the mean below 40)
    near(ent, want[1], extra=base * np.abs(want[1]).max() + 2.0 ** -18)


def make(seed, n, v, dtype, scale=2.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, v, generator=g) * scale
    t = torch.randint(0, v, (n,), generator=g)
    return x.to(dtype), t


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v,top", [
    (1, 1, 0), (1, 1, 1), (3, 2, 2), (2, 33, 32), (5, 257, 32), (1, 1000, 5), (9, 1024, 1),
    (4, 8191, 8), (23, 20001, 32), (1, 151936, 20), (2, 151936, 32), (200, 5003, 7),
    (400, 3001, 3), (700, 513, 32)])
def test_shapes(n, v, top, dtype):
    x, t = make(n * 1000 + v, n, v, dtype)
    check(x.to(DEV), t, top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_long_rows_and_many(dtype):
    x, t = make(3, 23, 151936, dtype)
    x[:, 1000] += 20
    check(x.to(DEV), t, 8)
    x, t = make(4, 700, 15193, dtype)       # one CTA a row
    check(x.to(DEV), t, 5)


@pytest.mark.parametrize("n", [2, 700])
@pytest.mark.parametrize("kind", ["equal", "ascending", "descending", "zeros", "two_values",
                                  "sawtooth"])
def test_orders_and_ties(kind, n):
    """Rows that collect more candidates than the buffer holds."""
    v = 20011
    i = torch.arange(v).float()
    x = {"equal": torch.full((v,), 3.25), "ascending": i / 1024, "descending": -i / 1024,
         "zeros": torch.where(torch.arange(v) % 2 == 0, 0.0, -0.0),
         "two_values": (torch.arange(v) % 3 == 1).float(), "sawtooth": (i % 97) + i / 1e5}[kind]
    x = x[None].repeat(n, 1)
    t = torch.arange(n) % v
    check(x.to(DEV), t, 32)
    check(x.to(DEV).to(torch.bfloat16), t, 9)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("masked", [-np.inf, "lowest"])
def test_masked_logits(dtype, masked):
    x, t = make(5, 6, 9001, dtype)
    low = torch.finfo(dtype).min if masked == "lowest" else -np.inf
    x[0, :9000] = low                # one left
    x[1, 3:] = low                   # three left, fewer than asked for
    x[2, ::2] = low
    x[3, 4000:8900] = low
    x[4, :] = low
    x[4, 8999] = -50.0
    t[0], t[1], t[2] = 9000, 1, 1
    check(x.to(DEV), t, 8)
    one = torch.full((1, 5000), float(torch.finfo(dtype).min), dtype=dtype)
    lp, ent, ids, tlp, _ = run(one.to(DEV), torch.tensor([7]), 4)      # uniform
    assert abs(ent[0] - np.log(5000)) < 1e-4 and ids[0].tolist() == [0, 1, 2, 3]


def test_rows_without_a_distribution():
    x, t = make(6, 5, 4000, torch.float32)
    x[0] = -np.inf
    x[1, 17] = np.nan
    x[2, 18] = np.inf
    lp, ent, ids, tlp, _ = run(x.to(DEV), t, 4)
    assert np.isnan(lp[:3]).all() and np.isnan(ent[:3]).all()
    assert ids[0].tolist() == [0, 1, 2, 3] and ((0 <= ids) & (ids < 4000)).all()
    want = OL.token_logprobs(x[3:].double().numpy(), t[3:].numpy(), 4)
    assert np.allclose(lp[3:], want[0], atol=1e-5) and np.array_equal(ids[3:], want[2])


def test_tokens_outside_the_vocabulary():
    x, _ = make(7, 4, 1000, torch.float32)
    lp, ent, ids, tlp, st = run(x.to(DEV), torch.tensor([5, -1, 1000, 999]), 2)
    assert st == api.DEV_BAD_TOKEN
    assert np.isnan(lp[1]) and np.isnan(lp[2]) and np.isfinite(lp[[0, 3]]).all()
    assert np.isfinite(ent).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (64, 3), (5, 2)])
def test_strided_and_unaligned_rows(dtype, pad, shift):
    n, v = 7, 4099
    x, t = make(8, n, v, dtype)
    buf = torch.full((n * (v + pad) + shift,), 50.0, dtype=dtype, device=DEV)
    view = buf[shift:].view(n, v + pad)[:, :v]
    view.copy_(x.to(DEV))
    check(view, t, 11)


def test_parts_left_out():
    x, t = make(9, 3, 2000, torch.bfloat16)
    x = x.to(DEV)
    full = run(x, t, 4)
    lp, ids = torch.empty(3, device=DEV), torch.empty(3, 4, dtype=torch.int32, device=DEV)
    api.token_logprobs(x, t.to(DEV, torch.int32), lp)
    assert np.array_equal(lp.cpu().numpy(), full[0])
    api.token_logprobs(x, None, None, None, ids)
    assert np.array_equal(ids.cpu().numpy(), full[2])
    api.token_logprobs(x[:0], t[:0].to(DEV, torch.int32), lp[:0])


def test_repeats_are_bit_equal_and_capture():
    x, t = make(10, 23, 50021, torch.bfloat16)
    x[:, 7000:9000] = 9.0       # many ties at the top
    xd, td = x.to(DEV), t.to(DEV, torch.int32)
    outs = (torch.empty(23, device=DEV), torch.empty(23, device=DEV),
            torch.empty(23, 32, dtype=torch.int32, device=DEV), torch.empty(23, 32, device=DEV))
    api.token_logprobs(xd, td, *outs)
    first = [o.clone() for o in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.token_logprobs(xd, td, *outs)
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, f in zip(outs, first):
            assert torch.equal(o, f)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("order", ["random", "ascending", "descending", "ties"])
@pytest.mark.parametrize("n,v,top", [(66, 100003, 32), (80, 60000, 20), (30, 200001, 32),
                                     (320, 50021, 32), (310, 90001, 7)])
def test_long_rows_of_many(n, v, top, order, dtype):
    # slices of many chunks: the bound of the alternatives is renewed several
    # times, and (ascending, ties) the candidates outgrow their buffer
    x, t = make(n + v, n, v, torch.float32)
    if order != "random":
        x = x.sort(dim=1, descending=order == "descending").values
    if order == "ties":
        x = x[:, torch.randperm(v, generator=torch.Generator().manual_seed(n))].clamp(max=2.0)
    check(x.to(dtype).to(DEV), t, top)
