"""Gradients of the weighted sum where some rows are named by no position."""
import pytest
import torch

from tests import _experts as X
from tests._gpu import TORCH

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def I8():
    import int8_quantized_linear_rowwise_amd as m
    return m


def littered(shape, dtype):
    """What the allocator gives out next for this shape holds NaN, not zeros."""
    junk = [torch.full(shape, float("nan"), dtype=dtype, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    del junk


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_positions_left_out_after_the_sort(I8, dt):
    """A choice taken out after the sort: its row, below the sort's last offset, gets a gradient of 0."""
    T, k, E, N = 60, 2, 4, 48
    off, _, pos = I8.expert_sort(X.choices(T, k, E, 1, 0.1).to(DEV), E)
    pos[torch.rand(T, k, device=DEV) < 0.3] = -1
    G = X.inputs(T, N, dt, 2, 0).to(DEV)
    gate = torch.rand(T, k, device=DEV)
    Y = torch.zeros((T * k, N), dtype=TORCH[dt], device=DEV, requires_grad=True)
    littered((T * k, N), TORCH[dt])
    I8.ExpertCombineFunction.apply(Y, pos, gate, None, off[-1:]).backward(G)
    want, slack = X.combine_gradient(G, pos, gate, T * k)
    X.check(Y.grad, want, X.rounded(want, slack, dt), "grad_Y")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,k,E,N", [(1, 2, 8, 256), (300, 2, 4, 1100), (129, 8, 16, 512), (20, 3, 5, 1023)])
def test_sum_gradient_of_the_sorts_positions(I8, dt, T, k, E, N):
    """To the last bit what expert_combine_backward gives, which takes positions that name no row twice."""
    off, _, pos = I8.expert_sort(X.choices(T, k, E, 3, 0.2).to(DEV), E)
    Y, G = X.inputs(T * k, N, dt, 1, 0).to(DEV).requires_grad_(), X.inputs(T, N, dt, 2, 0).to(DEV)
    G[:, ::7] = -0.0
    gate = torch.rand(T, k, device=DEV, requires_grad=True)
    I8.ExpertCombineFunction.apply(Y, pos, gate, None, off[-1:]).backward(G)
    gY, gg = I8.expert_combine_backward(G, pos, gate.detach(), Y.detach(), n_rows=off[-1:])
    assert torch.equal(Y.grad.view(torch.uint8), gY.view(torch.uint8)) and torch.equal(gate.grad, gg)


def test_no_choices_and_no_tokens(I8):
    """Nothing names a row: zeros."""
    for T, k in ((3, 0), (0, 2)):
        Y = torch.ones((5, 24), device=DEV, requires_grad=True)
        littered((5, 24), torch.float32)
        pos = torch.zeros((T, k), dtype=torch.int32, device=DEV)
        out = I8.ExpertCombineFunction.apply(Y, pos, None, None, None)
        out.backward(torch.ones_like(out))
        assert out.shape == (T, 24) and (Y.grad == 0).all()
