"""A mixture's layers through autograd, every stage held to its 64-bit form; many segments; long contractions."""
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


def token_gradient(G, CB, SCB, off, position, dt):
    """(x.grad, bound) where each row's gradient is rounded to the type and a token's rows are added in fp32."""
    rows, slack = X.backward(G, CB, SCB, off)
    row_bound = X.rounded(rows, slack, dt)
    T, k = position.shape
    y = torch.zeros((T, rows.shape[1]), dtype=X.d, device=G.device)
    bound, mag = torch.zeros_like(y), torch.zeros_like(y)
    for j in range(k):
        t = (position[:, j] >= 0).nonzero()[:, 0]
        r = position[t, j].long()
        y = y.index_add(0, t, rows[r])
        bound = bound.index_add(0, t, row_bound[r])
        mag = mag.index_add(0, t, rows[r].abs() + row_bound[r])
    return y, X.rounded(y, bound + k * 2.0 ** -24 * mag, dt)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,k,E,K,H", [(70, 2, 5, 96, 160), (300, 4, 16, 264, 136), (1, 2, 4, 512, 256),
                                       (4, 2, 3, 4096, 72), (600, 2, 3, 1040, 700)])
def test_mixture_stage_by_stage(I8, dt, T, k, E, K, H):
    """Sort, up projection with outlier columns, SiLU, down projection, weighted sum with a residual, and back: each
    stage from what the stage before really gave."""
    CBu, SCBu = X.weights(E, H, K, 1)
    CBd, SCBd = X.weights(E, K, H, 2)
    x = X.inputs(T, K, dt, 3, 3)
    gate = torch.rand((T, k), generator=torch.Generator().manual_seed(4))
    ids = X.choices(T, k, E, 5, 0.1)
    G = X.inputs(T, K, dt, 6, 0)
    CBu, SCBu, CBd, SCBd, x, gate, ids, G = (t.to(DEV) for t in (CBu, SCBu, CBd, SCBd, x, gate, ids, G))
    x.requires_grad_(), gate.requires_grad_()
    off, token, pos = I8.expert_sort(ids, E)
    h = I8.Int8ExpertsFunction.apply(x, CBu, SCBu, off, None, token, pos, 6.0)
    a = torch.nn.functional.silu(h)
    z = I8.Int8ExpertsFunction.apply(a, CBd, SCBd, off, None, None, None, 6.0)
    y = I8.ExpertCombineFunction.apply(z, pos, gate, x, off[-1:])
    for t in (h, a, z):
        t.retain_grad()
    y.backward(G)

    want, slack = X.forward(x.detach(), CBu, SCBu, off, None, token)
    X.check(h.detach(), want, X.rounded(want, slack, dt), "h")
    want, slack = X.forward(a.detach(), CBd, SCBd, off)
    X.check(z.detach(), want, X.rounded(want, slack, dt), "z")
    want, slack = X.combine(z.detach(), pos, gate.detach(), x.detach())
    X.check(y.detach(), want, X.rounded(want, slack, dt), "y")

    want, slack = X.combine_gradient(G, pos, gate.detach(), T * k)
    X.check(z.grad, want, X.rounded(want, slack, dt), "z.grad")
    _, want, slack = X.combine_backward(G, pos, gate.detach(), z.detach(), T * k)
    X.check(gate.grad, want, X.rounded(want, slack, "f32"), "gate.grad")
    want, slack = X.backward(z.grad, CBd, SCBd, off)
    X.check(a.grad, want, X.rounded(want, slack, dt), "a.grad")
    want, bound = token_gradient(h.grad, CBu, SCBu, off, pos, dt)
    # the residual's gradient is added to it in the type: one more rounding
    total = want + G.to(X.d)
    X.check(x.grad, total, X.rounded(total, bound, dt), "x.grad")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("k", [64, 65, 150])
def test_token_gradient_of_many_choices(I8, dt, k):
    """More rows a token than one weighted sum takes."""
    T, E, K, N = 20, 3, 72, 40
    CB, SCB = X.weights(E, N, K, 1)
    ids = X.choices(T, k, E, 2, 0.2)
    CB, SCB, ids = CB.to(DEV), SCB.to(DEV), ids.to(DEV)
    x, G = X.inputs(T, K, dt, 3).to(DEV).requires_grad_(), X.inputs(T * k, N, dt, 4, 0).to(DEV)
    off, token, pos = I8.expert_sort(ids, E)
    y = I8.Int8ExpertsFunction.apply(x, CB, SCB, off, None, token, pos, 6.0)
    y.backward(G)
    want, bound = token_gradient(G, CB, SCB, off, pos, dt)
    X.check(x.grad, want, bound, "x.grad")


# ---- segments -------------------------------------------------------------------------------------------------------


def segments(S, R, E, seed):
    """Offsets of S segments of very different lengths, many empty, with rows behind the last; experts among -1 .. E."""
    g = torch.Generator().manual_seed(seed)
    share = torch.rand(S, generator=g).pow(6) * (torch.rand(S, generator=g) < 0.8)
    share[S // 3] += 0.15 * share.sum()
    at = (share.cumsum(0) / share.sum() * (R - 9)).int()
    ids = torch.randint(-1, E + 1, (S,), generator=g).int()
    ids[S // 3] = 0
    return torch.cat([torch.zeros(1, dtype=torch.int32), at]), ids


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S", [254, 255, 256, 257, 600, 1024])
@pytest.mark.parametrize("R,K,N", [(900, 96, 40),            # tiles of 16 rows
                                   (12000, 272, 300), (12000, 271, 131),      # 128 x 128
                                   (11000, 1040, 300), (11000, 1041, 259)])   # 256 x 256
def test_products_of_many_segments(I8, dt, S, R, K, N):
    E, T = 4, 500
    CB, SCB = X.weights(E, N, K, 1)
    x = X.inputs(T, K, dt, 2)
    off, ids = segments(S, R, E, S)
    rows = torch.randint(-1, T + 1, (R,), generator=torch.Generator().manual_seed(3)).int()
    x, CB, SCB, off, ids, rows = (t.to(DEV) for t in (x, CB, SCB, off, ids, rows))
    out = torch.full((R, N), float("nan"), dtype=TORCH[dt], device=DEV)
    I8.expert_forward(x, CB, SCB, off, ids, rows, out=out)
    y, slack = X.forward(x, CB, SCB, off, ids, rows)
    X.check(out, y, X.rounded(y, slack, dt), "out")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S", [254, 255, 256, 257, 600, 1024])
@pytest.mark.parametrize("R,N,K", [(900, 96, 40), (12000, 264, 300), (12000, 263, 131),      # 128 x 128
                                   (11000, 600, 100), (11000, 601, 101)])                     # 256 x 256
def test_gradients_of_many_segments(I8, dt, S, R, N, K):
    E = 4
    CB, SCB = X.weights(E, N, K, 1)
    G = X.inputs(R, N, dt, 2, 0)
    off, ids = segments(S, R, E, S)
    G, CB, SCB, off, ids = (t.to(DEV) for t in (G, CB, SCB, off, ids))
    out = torch.full((R, K), float("nan"), dtype=TORCH[dt], device=DEV)
    I8.expert_backward(G, CB, SCB, off, ids, grad_X=out)
    y, slack = X.backward(G, CB, SCB, off, ids)
    X.check(out, y, X.rounded(y, slack, dt), "grad_X")


def test_more_experts_than_the_scan_holds(I8):
    """300 experts, each its own segment, through the sort: forward, gradient and sum."""
    T, k, E, K, N = 2000, 4, 300, 520, 264
    CB, SCB = (t.to(DEV) for t in X.weights(E, N, K, 1))
    x = X.inputs(T, K, "bf16", 2).to(DEV).requires_grad_()
    off, token, pos = I8.expert_sort(X.choices(T, k, E, 3, 0.1).to(DEV), E)
    G = X.inputs(T * k, N, "bf16", 4, 0).to(DEV)
    y = I8.Int8ExpertsFunction.apply(x, CB, SCB, off, None, token, pos, 6.0)
    y.backward(G)
    want, slack = X.forward(x.detach(), CB, SCB, off, None, token)
    X.check(y.detach(), want, X.rounded(want, slack, "bf16"), "y")
    want, bound = token_gradient(G, CB, SCB, off, pos, "bf16")
    X.check(x.grad, want, bound, "x.grad")


# ---- long contractions ----------------------------------------------------------------------------------------------


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,K,N", [(1, 11008, 96), (4, 11008, 136), (40, 11008, 264), (300, 11008, 520),
                                   (100, 4104, 72), (100, 5000, 72), (100, 8200, 136), (100, 16392, 40), (70, 32760, 24),
                                   (70, 33000, 24), (3, 8184, 40), (20, 8200, 40)])
def test_products_of_long_contractions(I8, dt, T, K, N):
    """Past what one launch, one wave a row or one workgroup a row quantizes, and rows that end in the middle of a piece
    of 16 codes."""
    E = 2
    CB, SCB = X.weights(E, N, K, 1)
    x = X.inputs(T, K, dt, 2, 5)
    off, token, _ = X.sort(X.choices(T, 2, E, 3, 0.1), E)
    x, CB, SCB, off, token = (t.to(DEV) for t in (x, CB, SCB, off, token))
    got = I8.expert_forward(x, CB, SCB, off, rows=token)
    y, slack = X.forward(x, CB, SCB, off, None, token)
    X.check(got, y, X.rounded(y, slack, dt), "out")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("R,N,K", [(1, 11008, 264), (16, 11008, 600), (500, 11008, 1028), (130, 11007, 259)])
def test_gradients_of_long_contractions(I8, dt, R, N, K):
    E = 2
    CB, SCB = X.weights(E, N, K, 1)
    G = X.inputs(R, N, dt, 2, 0)
    off = torch.tensor([0, R // 3, R], dtype=torch.int32)
    G, CB, SCB, off = (t.to(DEV) for t in (G, CB, SCB, off))
    got = I8.expert_backward(G, CB, SCB, off)
    y, slack = X.backward(G, CB, SCB, off)
    X.check(got, y, X.rounded(y, slack, dt), "grad_X")
