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


def planned_step(top=None):
    step = object.__new__(api.VerifyStep)      # (a step's buffers need a GPU)
    step.shape, step.int8, step.max_depth, step.top = (4, 6, 2, 64, 0, 200, 50), True, 8, top
    return step


@pytest.mark.parametrize("name,shape", [
    ("q", (3, 6, 64)), ("q", (5, 6, 64)), ("q", (4, 4, 64)), ("q", (4, 6, 128)),
    ("tree_k", (3, 2, 64)), ("tree_k", (4, 1, 64)), ("tree_v", (5, 2, 64)),
    ("tree_v", (4, 2, 128)), ("logits", (3, 50)), ("logits", (5, 50)), ("logits", (4, 49)),
    ("logits", (200,))])
def test_a_step_over_an_int8_cache_takes_what_it_is_planned_for(name, shape):
    """Fewer rows of logits than nodes would leave argmax and path of an
    earlier step in place, for the commit to follow."""
    shapes = {"q": (4, 6, 64), "tree_k": (4, 2, 64), "tree_v": (4, 2, 64), "logits": (4, 50)}
    shapes[name] = shape
    a = {k: OnDevice(torch.zeros(s, dtype=torch.bfloat16)) for k, s in shapes.items()}
    i32 = OnDevice(torch.zeros(4, dtype=torch.int32))
    with pytest.raises(api.DfvError, match=f"{name} .*planned"):
        planned_step().run(cpu_cache(), a["q"], a["tree_k"], a["tree_v"], i32, i32, a["logits"])


@pytest.mark.parametrize("name", ["parent", "tokens"])
def test_a_step_over_an_int8_cache_checks_before_it_launches(name):
    a = {"parent": OnDevice(torch.zeros(4, dtype=torch.int32)),
         "tokens": OnDevice(torch.zeros(4, dtype=torch.int32))}
    rows = OnDevice(torch.zeros(4, 2, 64, dtype=torch.bfloat16))
    for bad in (torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)):
        with pytest.raises(api.DfvError, match=name):
            planned_step().run(cpu_cache(), OnDevice(torch.zeros(4, 6, 64, dtype=torch.bfloat16)),
                               rows, rows, *{**a, name: OnDevice(bad)}.values(),
                               OnDevice(torch.zeros(4, 50)))


@pytest.mark.parametrize("fmt", ["int8", "q4_0", "f16"])
@pytest.mark.parametrize("top,vocab", [(33, 1000), (6, 5), (-1, 1000)])
def test_a_step_with_too_many_alternatives(top, vocab, fmt):
    """Refused when it is planned, not when a step has been committed."""
    with pytest.raises(api.DfvError, match="alternatives"):
        api.VerifyStep(4, 6, 2, 64, 0, 200, vocab, fmt=fmt, top=top, device="cpu")


@pytest.mark.parametrize("shape,dtype", [((4 * 50,), torch.float32), ((1, 4, 50), torch.bfloat16),
                                         ((5, 50), torch.float32), ((4, 50), torch.int16)])
def test_log_probabilities_of_whatever_logits_a_step_takes(shape, dtype, monkeypatch):
    """The other formats take n * vocab logits in any shape; the log
    probabilities come after the commit and must not refuse them then."""
    seen = []
    monkeypatch.setattr(api, "token_logprobs", lambda x, *a, **k: seen.append(x))
    step = planned_step(top=2)
    for name in ("argmax", "logprob", "entropy", "top_ids", "top_logprobs", "status"):
        setattr(step, name, None)
    x = torch.arange(torch.Size(shape).numel()).view(shape).to(dtype)
    step._logprobs(x, None)
    got = seen[0] if dtype != torch.int16 else seen[0].view(torch.int16)
    assert got.shape == (4, 50) and torch.equal(got, x.reshape(-1)[:200].view(4, 50))
    assert seen[0].dtype == (torch.bfloat16 if dtype == torch.int16 else dtype)
