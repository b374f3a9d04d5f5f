"""fp16 adapters: V and dV enter products as two fp16 values scaled by a power of
two of their own token. A token's output and input gradient do not depend on
its neighbours, however far apart their sizes lie, and keep the 17 bits of the
split."""
import pytest
import torch

from tests import _finetune as F
from tests.test_gpu_lora import I8, gpu  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu
KEYS = ("X", "A", "B", "scaling", "G")

# T, K, N, R: the forward in one launch, in two with 16-token tiles and with 64 (32 at rank 128) tokens; whole groups
# of columns and not; every rank class. The backward in tiles and in blocks of tiles.
CASES = [(16, 512, 192, 16), (40, 1024, 72, 24), (33, 1024, 192, 64), (20, 512, 136, 128), (48, 8192, 72, 16),
         (48, 4096, 128, 32), (30, 2048, 72, 64), (35, 1024, 128, 128), (1100, 512, 192, 16), (1100, 512, 72, 50),
         (1100, 320, 128, 128)]


def inputs(T, K, N, R, seed):
    """Every fifth row is large in all features, the others small and in one feature only: V and dV of neighbours lie
    2^26 to 2^31 apart. All values are fp16's normal ones. The large rows' outputs are beyond fp16."""
    c = F.lora_inputs("f16", T, K, N, R, 1, seed)
    g = torch.Generator().manual_seed(seed + 50)
    large = torch.arange(T) % 5 == 2
    for k, n in (("X", K), ("G", N)):
        x = torch.randn((T, n), generator=g).clamp(-4, 4) * 2.0 ** 12
        at = torch.randint(0, n, (T,), generator=g)
        one = torch.zeros((T, n))
        one[torch.arange(T), at] = (1 + torch.rand(T, generator=g)) * 2.0 ** -13
        c[k] = torch.where(large[:, None], x, one).to(torch.float16)
    c["scaling"] = torch.tensor([4096.0])
    return c, large


@pytest.mark.parametrize("T,K,N,R", CASES)
def test_each_token_for_itself(I8, T, K, N, R):  # noqa: F811
    print(f"\n  [T={T} K={K} N={N} R={R}]", flush=True)
    c, large = inputs(T, K, N, R, 3)
    d = {k: gpu(c[k]) for k in KEYS}

    def calls(d):
        out, V = I8.lora_forward(d["X"], d["A"], d["B"], d["scaling"], with_v=True)
        gX, _, _ = I8.lora_backward(d["G"], d["X"], V, d["A"], d["B"], d["scaling"])
        return out, gX, V

    out, gX, V = calls(d)
    alone = dict(d, X=torch.where(large[:, None].cuda(), 0.0, d["X"]), G=torch.where(large[:, None].cuda(), 0.0, d["G"]))
    out1, gX1, _ = calls(alone)
    torch.cuda.synchronize()
    small = ~large
    y, lim, v64, vlim = F.lora_forward64(c, "f16", [(0, T, 0)], with_base=False)
    ratio = v64[large].abs().amax() / v64[small].abs().amax(1).min()
    assert ratio > 2.0 ** 26, ratio
    F.assert_within(V[small.cuda()], v64[small], vlim[small], "V")
    assert y[small].abs().max() < 6e4
    F.assert_within(out[small.cuda()], y[small], lim[small], "out")
    (w, e), _, _ = F.lora_backward64(c, "f16", [(0, T, 0)], with_base=False)
    assert w[small].abs().max() < 6e4
    F.assert_within(gX[small.cuda()], w[small], e[small], "grad_X")
    assert torch.equal(out[small.cuda()], out1[small.cuda()]) and torch.equal(gX[small.cuda()], gX1[small.cuda()])


@pytest.mark.parametrize("T,K,N,R", CASES)
def test_sums_over_tokens_of_very_different_sizes(I8, T, K, N, R):  # noqa: F811
    """grad_A and grad_B, where one sum meets values of many tokens: besides the split's 2^-17, each value of dV (V) may
    be off by 2^-39 of the largest. The large rows are zero in half the features, where that can be seen."""
    print(f"\n  [T={T} K={K} N={N} R={R}]", flush=True)
    c, large = inputs(T, K, N, R, 4)
    for k, n in (("X", K), ("G", N)):
        c[k][large, :n // 2] = 0
    c["scaling"] = torch.tensor([1.0])
    d = {k: gpu(c[k]) for k in KEYS}
    _, V = I8.lora_forward(d["X"], d["A"], d["B"], d["scaling"], with_v=True)
    _, gA, gB = I8.lora_backward(d["G"], d["X"], V, d["A"], d["B"], d["scaling"])
    torch.cuda.synchronize()
    X, A, B, G = (c[k].double() for k in ("X", "A", "B", "G"))
    _, (wA, eA), (wB, eB) = F.lora_backward64(c, "f16", [(0, T, 0)], with_base=False)
    v, dv = X @ A[0].t(), G @ B[0]
    eA = eA + 1.01 * 2.0 ** -39 * dv.abs().max() * X.abs().sum(0)[None, None, :]
    eB = eB + 1.01 * 2.0 ** -39 * v.abs().max() * G.abs().sum(0)[None, :, None]
    for name, got, want, lim in (("grad_A", gA, wA, eA), ("grad_B", gB, wB, eB)):
        near = want.abs() + lim < 65504
        assert near.double().mean() > 0.4
        F.assert_within(torch.where(near, got.cpu().double(), 0.0), torch.where(near, want, 0.0), lim, name)
