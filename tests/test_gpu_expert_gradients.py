"""Gradients of the weighted sum for positions of any kind: rows named several times, by none, and positions changed
after the sort."""
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


def anyhow(kind, T, k, R, seed):
    """Positions: repeated at random, all the same, the first and the last of many alike, in pairs, or a sort's with
    some left out afterwards."""
    g = torch.Generator().manual_seed(seed)
    if kind == "random":
        pos = torch.randint(-2, R + 3, (T, k), generator=g)
    elif kind == "one row":
        pos = torch.full((T, k), R - 1)
    elif kind == "far":
        pos = torch.arange(T * k).view(T, k) % R
        pos[-1, -1] = pos[0, 0] = 1 % R
    elif kind == "pairs":
        pos = torch.arange(T * k).view(T, k) // 2 * 2 % max(R, 1)
    else:
        pos = torch.randperm(T * k, generator=g).view(T, k)
        pos[torch.rand((T, k), generator=g) < 0.3] = -1
    return pos.int()


KINDS = ["random", "one row", "far", "pairs", "left out"]
SIZES = [(1, 2, 8), (40, 3, 72), (33, 5, 1), (700, 2, 1100), (90, 8, 1023), (25, 4, 4100), (300, 64, 16)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,k,N", SIZES)
@pytest.mark.parametrize("gated,with_n_rows", [(True, True), (False, False)])
def test_sum_gradient_of_any_positions(I8, dt, kind, T, k, N, gated, with_n_rows):
    R = T * k
    pos = anyhow(kind, T, k, R, 3).to(DEV)
    g = torch.Generator().manual_seed(4)
    Y, G = (torch.randn(s, generator=g).to(TORCH[dt]).to(DEV) for s in ((R, N), (T, N)))
    gate = torch.rand((T, k), generator=g).to(DEV) if gated else None
    wY, slack = X.combine_gradient(G, pos, gate, R)
    _, wg, gslack = X.combine_backward(G, pos, gate, Y, R)
    got = []
    for _ in range(2):
        Yr = Y.clone().requires_grad_()
        gr = gate.clone().requires_grad_() if gated else None
        n_rows = torch.full((1,), R, dtype=torch.int32, device=DEV) if with_n_rows else None
        out = I8.ExpertCombineFunction.apply(Yr, pos, gr, None, n_rows)
        littered((R, N), TORCH[dt])
        out.backward(G)
        X.check(Yr.grad, wY, X.rounded(wY, slack, dt), "grad_Y")
        if gated:
            X.check(gr.grad, wg, X.rounded(wg, gslack, "f32"), "grad_gate")
        got.append(Yr.grad)
    assert torch.equal(*got)


def test_sum_gradient_of_repeats_far_apart(I8):
    """160000 choices of which the first and the last name one row, and one in a thousand another."""
    T, k, N = 20000, 8, 40
    pos = torch.randperm(T * k, generator=torch.Generator().manual_seed(1)).int()
    pos[-1] = pos[0]
    pos[::1000] = 77
    pos = pos.view(T, k).to(DEV)
    G = X.inputs(T, N, "bf16", 2, 0).to(DEV)
    gate = torch.rand(T, k, device=DEV)
    Y = torch.zeros((T * k, N), dtype=torch.bfloat16, device=DEV, requires_grad=True)
    littered((T * k, N), torch.bfloat16)
    I8.ExpertCombineFunction.apply(Y, pos, gate, None, None).backward(G)
    want, slack = X.combine_gradient(G, pos, gate, T * k)
    X.check(Y.grad, want, X.rounded(want, slack, "bf16"), "grad_Y")


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


def test_any_positions_into_given_rows(I8):
    """grad_Y and the workspace are the caller's: every row is written, nothing beside them is."""
    G = torch.ones((2, 24), device=DEV)
    pos = torch.tensor([[4, 1], [1, 9]], dtype=torch.int32, device=DEV)
    whole = torch.full((10, 24), 7.0, device=DEV)
    ws = torch.full((64,), 9, dtype=torch.uint8, device=DEV)
    I8.expert_combine_backward(G, pos, None, with_grad_gate=False, rows=6, grad_Y=whole[2:8], any_positions=True,
                               workspace=ws[4:52])
    assert whole[:, 5].tolist() == [7, 7, 0, 2, 0, 0, 1, 0, 7, 7]
    assert (ws[:4] == 9).all() and (ws[52:] == 9).all()


def test_any_positions_replayed(I8):
    """Captured once, replayed with other positions and eager work between: bit-identical to the eager call."""
    T, k, N = 200, 4, 264
    R = T * k
    G, Y = X.inputs(T, N, "bf16", 1, 0).to(DEV), X.inputs(R, N, "bf16", 2, 0).to(DEV)
    pos, gate = anyhow("random", T, k, R, 3).to(DEV), torch.rand(T, k, device=DEV)

    def step():
        return I8.expert_combine_backward(G, pos, gate, Y, any_positions=True)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i, kind in enumerate(KINDS):
        pos.copy_(anyhow(kind, T, k, R, 10 + i))
        G.copy_(X.inputs(T, N, "bf16", 20 + i, 0))
        torch.cuda.synchronize()
        graph.replay()
        there = [o.clone() for o in outs]
        here = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(here, there)), kind


@pytest.mark.parametrize("T,N", [(1 << 24, 1), ((1 << 20) + 3, 2048)])
def test_any_positions_of_very_many_tokens(I8, T, N):
    """The most tokens there can be, and more workgroups than one axis of the grid is given; the last two tokens name
    one row, so that the first token's row is named by none."""
    pos = torch.arange(T, dtype=torch.int32, device=DEV).view(T, 1).flip(0)
    pos[-1] = 1
    G = torch.ones((T, N), dtype=torch.bfloat16, device=DEV)
    gate = torch.full((T, 1), 0.5, device=DEV)
    gY, none = I8.expert_combine_backward(G, pos, gate, rows=T, with_grad_gate=False, any_positions=True)
    assert none is None and (gY[0] == 0).all() and (gY[1] == 1).all() and bool((gY[2:] == 0.5).all())
