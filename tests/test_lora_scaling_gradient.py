"""The factors of the adapters are not trained: a gradient for them is refused instead of silently left out."""
import pytest
import torch

from tests._stub_gpu import L, stub  # noqa: F401  (fixtures)


def call(I8, scaling):
    x = torch.zeros(4, 16, dtype=torch.float16, requires_grad=True)
    CB, SCB = torch.zeros(6, 16, dtype=torch.int8), torch.ones(6)
    A, B = torch.zeros(2, 8, 16, dtype=torch.float16), torch.zeros(2, 6, 8, dtype=torch.float16)
    return I8.Int8LoraFunction.apply(x, CB, SCB, None, A, B, scaling, None, None, 6.0)


def test_a_gradient_for_scaling_is_refused(stub):  # noqa: F811
    y = call(stub.I8, torch.ones(2, requires_grad=True))
    launched = len(stub.seen)
    with pytest.raises(ValueError, match="scaling"):
        y.sum().backward()
    assert len(stub.seen) == launched       # before anything of the backward ran
    call(stub.I8, torch.ones(2)).sum().backward()
    with torch.no_grad():                   # serving with factors that say they require a gradient
        call(stub.I8, torch.ones(2, requires_grad=True))
    assert len(stub.seen) == launched + 4 + 2
