"""GPU parity of layer norm and its gradient against the plain 64-bit forms
(tests/_finetune.py derives each element's bound)."""
import pytest
import torch

from tests import _finetune as F

pytestmark = pytest.mark.gpu
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")]


@pytest.fixture(scope="module")
def I8():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import int8_quantized_linear_rowwise_amd as I8
    return I8


def inputs(dt, wdt, T, C, seed, shift=0.3):
    X = (F.randn((T, C), "f32", seed) + shift).to(F.DT[dt])
    if C > 4:
        X[:, seed % C] *= 20
    w = (1 + 0.2 * F.randn((C,), "f32", seed + 1)).to(F.DT[wdt])
    return X, w, F.randn((C,), wdt, seed + 2, 0.2), F.randn((T, C), dt, seed + 3, 0.1)


def check(I8, dt, wdt, T, C, seed=1, with_bias=True, eps=1e-5, shift=0.3):
    what = f"[{dt} {wdt} T={T} C={C}]"
    print("\n  " + what, flush=True)
    X, w, b, G = inputs(dt, wdt, T, C, seed, shift)
    b = b if with_bias else None
    Xc, wc, Gc = X.cuda(), w.cuda(), G.cuda()
    y, mean, rstd = I8.layer_norm_forward(Xc, wc, b.cuda() if with_bias else None, eps)
    torch.cuda.synchronize()
    for name, t, (want, lim) in zip(("out", "mean", "rstd"), (y, mean, rstd), F.norm64(X, w, b, eps, dt)):
        F.assert_within(t, want, lim, f"{what} {name}")
    got = I8.layer_norm_backward(Gc, Xc, mean, rstd, wc)
    torch.cuda.synchronize()
    for name, t, (want, lim) in zip(("grad_X", "grad_weight", "grad_bias"), got,
                                    F.norm_backward64(G, X, mean.cpu(), rstd.cpu(), w, dt, wdt)):
        F.assert_within(t, want, lim, f"{what} {name}")


SIZES = [(1, 1), (3, 2), (5, 7), (1, 64), (2, 257), (70, 33), (33, 1000), (17, 1024), (9, 1001), (300, 264), (7, 4096),
         (40, 4104), (5, 8192), (3, 11008), (4, 12345), (2, 16384), (3, 20000), (1, 40007), (1500, 72), (600, 2056)]


@pytest.mark.parametrize("dt,wdt", TYPES)
@pytest.mark.parametrize("T,C", SIZES)
def test_sizes(I8, dt, wdt, T, C):
    check(I8, dt, wdt, T, C)


@pytest.mark.parametrize("dt,wdt", TYPES)
def test_without_bias_and_far_mean(I8, dt, wdt):
    check(I8, dt, wdt, 20, 520, with_bias=False)
    # a mean far over the spread: the variance comes from differences to it, not from squares
    check(I8, dt, wdt, 20, 520, shift=100.0)
    check(I8, dt, wdt, 20, 520, eps=0.0)


@pytest.mark.parametrize("dt,wdt", TYPES)
def test_wide_rows(I8, dt, wdt):
    check(I8, dt, wdt, 1, 262144)


def test_constant_and_not_finite_rows(I8):
    X = torch.ones((6, 520), dtype=torch.bfloat16, device="cuda:0")
    X[2], X[3, 5], X[4, 7] = 0.0, float("inf"), float("nan")
    X[5] = torch.randn(520, device="cuda:0").to(torch.bfloat16)
    w, b = torch.full((520,), 2.0, device="cuda:0"), torch.full((520,), 0.5, device="cuda:0")
    y, mean, rstd = I8.layer_norm_forward(X, w, b)
    assert (y[:3] == 0.5).all() and torch.isnan(y[3:5]).all() and torch.isfinite(y[5]).all()
    assert mean[0] == 1 and mean[2] == 0 and torch.isfinite(rstd[:3]).all()
    G = torch.randn(6, 520, device="cuda:0").to(torch.bfloat16)
    gX, _, gb = I8.layer_norm_backward(G, X, mean, rstd, w)
    assert torch.isfinite(gX[:3]).all() and torch.isnan(gX[3:5]).all() and torch.isfinite(gX[5]).all()
    assert torch.isfinite(gb).all()


def test_no_rows(I8):
    X = torch.zeros((0, 72), dtype=torch.float16, device="cuda:0")
    w = torch.ones(72, device="cuda:0")
    y, mean, rstd = I8.layer_norm_forward(X, w)
    gw, gb = torch.full_like(w, 7), torch.full_like(w, 7)
    gX, _, _ = I8.layer_norm_backward(X, X, mean, rstd, w, grad_weight=gw, grad_bias=gb)
    torch.cuda.synchronize()
    assert y.shape == gX.shape == (0, 72) and not gw.any() and not gb.any()
    E = torch.zeros((5, 0), dtype=torch.float16, device="cuda:0")
    assert I8.layer_norm_forward(E, w[:0])[0].shape == (5, 0)


@pytest.mark.parametrize("dt,wdt", TYPES)
@pytest.mark.parametrize("T,C", [(50, 520), (5, 4096), (3, 20000)])
def test_in_place_parts_and_views(I8, dt, wdt, T, C):
    X, w, b, G = (t.cuda() for t in inputs(dt, wdt, T, C, 4))
    y, mean, rstd = I8.layer_norm_forward(X, w, b)
    Z = X.clone()
    assert I8.layer_norm_forward(Z, w, b, out=Z)[0] is Z and torch.equal(Z, y)
    full = I8.layer_norm_backward(G, X, mean, rstd, w)
    for i, want in enumerate(full):
        on = [j == i for j in range(3)]
        got = I8.layer_norm_backward(G, X, mean, rstd, w, *on)
        assert torch.equal(got[i], want) and all(got[j] is None for j in range(3) if j != i)
    Z = G.clone()
    I8.layer_norm_backward(Z, X, mean, rstd, w, True, False, False, grad_X=Z)
    assert torch.equal(Z, full[0])

    def shift(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
        s[1:] = t.reshape(-1)
        return s[1:].view(t.shape)

    ys, ms, rs = I8.layer_norm_forward(shift(X), shift(w), shift(b), out=shift(y))
    (yw, ylim), _, _ = F.norm64(X.cpu(), w.cpu(), b.cpu(), 1e-5, dt)
    F.assert_within(ys, yw, ylim, "shifted out")
    got = I8.layer_norm_backward(shift(G), shift(X), shift(mean), shift(rstd), shift(w), grad_X=shift(X))
    for name, t, (want, lim) in zip(("grad_X", "grad_weight", "grad_bias"), got,
                                    F.norm_backward64(G.cpu(), X.cpu(), mean.cpu(), rstd.cpu(), w.cpu(), dt, wdt)):
        F.assert_within(t, want, lim, "shifted " + name)


def test_stream_graph_and_determinism(I8):
    T, C = 900, 1032
    X, w, b, G = (t.cuda() for t in inputs("bf16", "f32", T, C, 5))

    def calls():
        y, mean, rstd = I8.layer_norm_forward(X, w, b)
        return (y, mean, rstd) + I8.layer_norm_backward(G, X, mean, rstd, w)

    want = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = calls()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = calls()
    for seed in (6, 7, 8):
        X2, _, _, G2 = inputs("bf16", "f32", T, C, seed)
        X.copy_(X2)
        G.copy_(G2)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(held, calls())), seed


def test_module_and_differences(I8):
    """The module's gradients are the calls' bits; fp32 gradients against central differences of the kernel."""
    ln = I8.LayerNorm(24, device="cuda:0")
    with torch.no_grad():
        ln.weight.copy_(1 + 0.2 * F.randn((24,), "f32", 30))
        ln.bias.copy_(F.randn((24,), "f32", 31))
    x = F.randn((2, 3, 24), "f32", 32).cuda().requires_grad_(True)
    g = F.randn((2, 3, 24), "f32", 33).cuda()
    ln(x).backward(g)
    X, G = x.detach().reshape(6, 24), g.reshape(6, 24)
    _, mean, rstd = I8.layer_norm_forward(X, ln.weight.detach(), ln.bias.detach())
    gX, gw, gb = I8.layer_norm_backward(G, X, mean, rstd, ln.weight.detach())
    assert torch.equal(x.grad.reshape(6, 24), gX) and torch.equal(ln.weight.grad, gw) and torch.equal(ln.bias.grad, gb)

    def loss(X, w):
        return float((I8.layer_norm_forward(X, w, ln.bias.detach())[0].double() * G.double()).sum())

    h = 2.0 ** -8
    # second-order remainder of the norm (third derivative times h^2 / 6, at most about 10 h^2) and fp32's rounding
    # of the outputs, about 30 u over 144 values of size 3 with factors of size 1, over h
    lim = 10 * h * h * 10 + 30 * F.U * 144 * 3 / h
    w = ln.weight.detach()
    for t, grad, which in ((X, gX, 0), (w, gw, 1)):
        for i in range(0, t.numel(), 5):
            up, dn = t.clone(), t.clone()
            up.view(-1)[i] += h
            dn.view(-1)[i] -= h
            d = float(up.view(-1)[i]) - float(dn.view(-1)[i])
            diff = loss(up, w) - loss(dn, w) if which == 0 else loss(X, up) - loss(X, dn)
            assert abs(diff / d - float(grad.view(-1)[i])) <= lim, (which, i)


def test_second_derivatives_are_refused(I8):
    """The gradients are not differentiable again, and say so."""
    x = torch.randn(4, 32, device="cuda:0", requires_grad=True)
    y = I8.LayerNorm(32, device="cuda:0")(x)
    (g,) = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


@pytest.mark.parametrize("C,T", [(64, 64), (64, 65), (128, 64), (1024, 8), (1024, 9), (2048, 4), (2048, 5), (4096, 2),
                                 (4096, 3), (16384, 1), (16384, 2), (1024, 16), (1024, 17), (4096, 4), (4096, 5),
                                 (8192, 2), (8192, 3)])
def test_few_rows(I8, C, T):
    """Both sides of where one workgroup takes all rows."""
    check(I8, "bf16", "f32", T, C)
