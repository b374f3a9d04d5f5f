"""What a gradient norm's plan checks and holds on the host."""
import pytest
import torch

from tests._stub_gpu import stub  # noqa: F401  (fixture)
from tests.test_abi import L  # noqa: F401  (fixture: builds the library if it is missing)


@pytest.fixture
def calls(stub, L, monkeypatch):  # noqa: F811
    seen = []
    monkeypatch.setattr(L.lib, "int8_grad_norm", lambda *a: seen.append(a) or 0)
    return seen


@pytest.mark.parametrize("parts", [
    [(0, 60), (59, 100)], [(59, 100), (0, 60)], [(0, 100), (40, 41)], [(40, 41), (0, 100)], [(0, 100), (0, 1)],
    [(0, 30), (70, 100), (29, 71)], [(5, 9), (5, 9)],
])
def test_clipping_refuses_gradients_that_overlap(stub, calls, parts):  # noqa: F811
    """Two workgroups would read, scale and write the same values."""
    flat = torch.zeros(100)
    plan = stub.I8.GradNormPlan([flat[a:b] for a, b in parts])
    plan.norm(1.0)                           # reading twice is fine
    assert len(calls) == 1
    for _ in range(2):
        with pytest.raises(ValueError, match="twice"):
            plan.clip(1.0)
    assert len(calls) == 1
    p = []
    for a, b in parts:
        p.append(torch.nn.Parameter(torch.zeros(b - a)))
        p[-1].grad = flat[a:b]
    with pytest.raises(ValueError, match="twice"):
        stub.I8.clip_grad_norm_(p, 1.0)


def test_neighbours_do_not_overlap(stub, calls):  # noqa: F811
    flat, half = torch.zeros(100), torch.zeros(100, dtype=torch.bfloat16)
    stub.I8.GradNormPlan([flat[50:], flat[:50], flat[20:20], half[:1], half[1:], half[7:7]]).clip(1.0)
    assert len(calls) == 1


@pytest.mark.parametrize("move", ["data", "set_"])
def test_a_plan_holds_the_memory_that_it_names(stub, calls, move):  # noqa: F811
    """A gradient that is given other memory later: the plan's calls go on with what it was laid out for, which nobody
    else has been given meanwhile."""
    g = [torch.zeros(300), torch.zeros(40)]
    plan = stub.I8.GradNormPlan(g)
    memory = g[0].untyped_storage()._weak_ref()
    address = g[0].data_ptr()
    if move == "data":
        g[0].data = torch.ones(300)
    else:
        g[0].set_(torch.ones(300))
    plan.norm(1.0)
    assert calls[-1][0][0] == address and not torch.UntypedStorage._expired(memory)
    del plan
    calls.clear()
    assert torch.UntypedStorage._expired(memory)


@pytest.mark.parametrize("how", ["deepcopy", "copy", "pickle"])
def test_a_copied_plan_names_its_own_gradients(stub, calls, how):  # noqa: F811
    import copy
    import pickle
    g = [torch.arange(300.0), torch.zeros(40)]
    plan = stub.I8.GradNormPlan(g)
    plan.norm(1.0)
    other = {"deepcopy": copy.deepcopy, "copy": copy.copy,
             "pickle": lambda p: pickle.loads(pickle.dumps(p))}[how](plan)
    other.norm(1.0)
    mine, theirs = calls[-2][0], calls[-1][0]
    held = other._keep[0]
    assert [theirs[0], theirs[3]] == [t.data_ptr() for t in held] and torch.equal(held[0], g[0])
    assert (mine[0] == theirs[0]) == (how == "copy")
