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
