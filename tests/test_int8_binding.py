"""Arguments that the binding of the 8-bit cache, its steps and the log
probabilities refuses by itself (CPU: no launch is reached)."""

import pytest
import torch

from tree_verify_attention_gb300 import api


def cpu_cache(capacity=200):
    return api.Int8Cache(2, 64, capacity, device="cpu")


@pytest.mark.parametrize("at", [-1, -2, 201, 1 << 31, 1 << 32, (1 << 32) + 5, -(1 << 32)])
def test_positions_outside_the_cache(at):
    """A negative one is not `the committed length`, and a large one is not
    cut to 32 bits."""
    c, rows = cpu_cache(), torch.zeros(3, 2, 64)
    for call in (lambda: c.append(rows, rows, at=at), lambda: c.truncate(at),
                 lambda: c.fill(rows.transpose(0, 1), rows.transpose(0, 1), pos0=at),
                 lambda: c.read(at, 3, rows, rows)):
        with pytest.raises(api.DfvError, match="outside"):
            call()


def test_reads_past_the_capacity():
    c, rows = cpu_cache(), torch.zeros(3, 2, 64)
    for pos, n in ((198, 3), (0, 201), (0, -1), (5, 1 << 32)):
        with pytest.raises(api.DfvError, match="outside"):
            c.read(pos, n, rows, rows)


class OnDevice:
    """A host tensor that says it is on the GPU (nothing may be launched)."""

    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.mark.parametrize("ids,tlp", [(0, 5), (5, 0), (3, 5), (5, 3)])
def test_alternatives_of_two_widths(ids, tlp):
    """Also where one has no columns: a view of none still has an address."""
    n, v = 3, 40
    store = torch.zeros(n, 8, dtype=torch.int32)
    ids = OnDevice(store[:, :ids].contiguous() if ids else store[:, :0])
    tlp = OnDevice(torch.zeros(n, tlp))
    with pytest.raises(api.DfvError, match="the same K"):
        api.token_logprobs(OnDevice(torch.zeros(n, v)), None, None, None, ids, tlp)
