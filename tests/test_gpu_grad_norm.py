"""The gradient norm and clipping on the GPU against their plain 64-bit form."""
import math

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


def grads(sizes, dt, seed=1, scale=1e-3):
    g = torch.Generator().manual_seed(seed)
    kinds = ["f32", "f16", "bf16"] if dt == "mixed" else [dt]
    return [(torch.randn(n, generator=g) * scale).to(TORCH[kinds[i % len(kinds)]]).to(DEV) for i, n in enumerate(sizes)]


def near(got, want):
    """One rounding to fp32 of a value formed in 64 bits (whose own error is far below)."""
    return abs(float(got) - want) <= 2.0 ** -23 * abs(want)


LISTS = [[1], [0, 5, 0], [8191, 8192, 8193], [31] * 200, [100000, 1, 7, 65536], [3] * 161 + [0] * 160 + [9],
         [20_000_003], [131072], [131073], [5] * 16, [5] * 17, [0] * 290, [0] * 285 + [4],
         [3] * 281 + [0] * 280 + [9], [4, 16384] * 150]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", LISTS)
@pytest.mark.parametrize("kind", [2, math.inf])
def test_norm_and_clip(I8, dt, sizes, kind):
    g = grads(sizes, dt)
    plan = I8.GradNormPlan(g)
    full, _ = X.grad_norm(g, math.inf, kind)
    for top, c in ((None, None), (full / 3, None), (full * 2, 0.5), (full / 8, 0.25), (0.0, None)):
        want, factor = X.grad_norm(g, math.inf if top is None else top, kind, 1.0 if c is None else c)
        scale = None if c is None else torch.tensor(c, device=DEV)
        norm, f, bad = plan.norm(top, kind, scale)
        assert near(norm, want) and near(f, factor) and float(bad) == 0, (top, c)
        again = plan.norm(top, kind, scale)
        assert all(torch.equal(a, b) for a, b in zip((norm, f, bad), again))
    before = [x.clone() for x in g]
    norm, f, bad = plan.clip(full / 3, kind)
    assert near(norm, full)
    for a, b in zip(g, before):
        assert torch.equal(a, (b.float() * f).to(b.dtype))


def test_clip_writes_nothing_within_the_norm(I8):
    g = grads([1000, 17], "bf16")
    before = [x.clone() for x in g]
    norm, f, _ = I8.GradNormPlan(g).clip(1e9)
    assert float(f) == 1.0 and all(torch.equal(a, b) for a, b in zip(g, before))


def test_unaligned_and_odd(I8):
    raw = grads([50001], "f16")[0]
    g = [raw[1:40000], raw[40003:]]
    want, _ = X.grad_norm(g)
    norm, _, _ = I8.GradNormPlan(g).norm()
    assert near(norm, want)
    keep = raw.clone()
    _, f, _ = I8.GradNormPlan(g).clip(want / 2)
    assert torch.equal(raw[1:40000], (keep[1:40000].float() * f).half())
    assert raw[0] == keep[0] and torch.equal(raw[40000:40003], keep[40000:40003])


@pytest.mark.parametrize("dt,value", [("f32", 3e38), ("f32", 1e-30), ("bf16", 1e38), ("bf16", 1e-38), ("f16", 60000.0)])
def test_far_magnitudes(I8, dt, value):
    """Squares that fp32 does not hold."""
    g = [torch.full((n,), value, device=DEV).to(TORCH[dt]) for n in (3, 7)]
    for kind in (2, math.inf):
        want, _ = X.grad_norm(g, math.inf, kind)
        norm, _, bad = I8.GradNormPlan(g).norm(None, kind)
        if want > 3.4028234e38:
            assert math.isinf(float(norm)) and float(bad) == 1
        else:
            assert near(norm, want) and float(bad) == 0


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", [2, math.inf])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_not_finite(I8, dt, kind, value):
    g = grads([5000, 9], dt)
    g[0][4321] = value
    norm, f, bad = I8.GradNormPlan(g).norm(1.0, kind)
    assert float(bad) == 1
    if math.isnan(value):
        assert math.isnan(float(norm)) and math.isnan(float(f))
    else:
        assert math.isinf(float(norm)) and float(f) == 0
    norm, f, bad = I8.GradNormPlan(g).norm(None, kind)
    assert float(bad) == 1 and float(f) == 1


def test_nan_beside_infinity(I8):
    for where in ((0, 1), (1, 0)):
        g = torch.zeros(2, 4000, device=DEV)
        g[where[0], 3], g[where[1], 7] = math.inf, math.nan
        for kind in (2, math.inf):
            assert math.isnan(float(I8.GradNormPlan([g[0], g[1]]).norm(1.0, kind)[0]))


def test_clip_function_and_optimizer(I8):
    p = [torch.nn.Parameter(x) for x in grads([300, 40, 5], "bf16", 1, 1.0)]
    for q, x in zip(p[:2], grads([300, 40], "bf16", 2)):
        q.grad = x
    want, _ = X.grad_norm([p[0].grad, p[1].grad])
    keep = p[0].grad.clone()
    opt = I8.AdamW(p, lr=0.1)
    norm, f, bad = opt.grad_norm(want / 2)
    assert near(norm, want) and f.shape == () and f.dtype == torch.float32
    opt.step(grad_scale=f, found_inf=bad)
    got = I8.clip_grad_norm_(p, want / 2)
    assert near(got, want) and torch.equal(p[0].grad, (keep.float() * f).to(keep.dtype))
    p[0].grad[3] = math.inf
    before = [q.detach().clone() for q in p]
    _, f, bad = opt.grad_norm(1.0)
    opt.step(grad_scale=f, found_inf=bad)
    assert all(torch.equal(q, b) for q, b in zip(p, before))          # the step is left out


def test_refusals(I8):
    g = grads([100], "f32")[0]
    with pytest.raises(ValueError, match="twice"):
        I8.GradNormPlan([g, g]).clip(1.0)
    I8.GradNormPlan([g, g]).norm(1.0)
    with pytest.raises(ValueError, match="contiguous"):
        I8.GradNormPlan([g.view(10, 10).t()])
    with pytest.raises(TypeError):
        I8.GradNormPlan([g.double()])
    with pytest.raises(ValueError, match="grad_scale"):
        I8.GradNormPlan([g]).norm(1.0, grad_scale=torch.ones(2, device=DEV))
    with pytest.raises(ValueError):
        I8.GradNormPlan([g, torch.zeros(3)])
    with pytest.raises(ValueError, match="workspace"):
        I8.GradNormPlan([torch.zeros(1 << 20, device=DEV)]).norm(
            1.0, workspace=torch.zeros(4, dtype=torch.uint8, device=DEV))


def test_replays(I8):
    """A captured norm, clipping and step: replays read the gradients and the scale that the buffers then hold."""
    p = [torch.nn.Parameter(x) for x in grads([5000, 300], "bf16", 1, 1.0)]
    for q, x in zip(p, grads([5000, 300], "bf16", 2)):
        q.grad = x
    q2 = [torch.nn.Parameter(q.detach().clone()) for q in p]
    for a, b in zip(q2, p):
        a.grad = b.grad.clone()
    opt, ref = I8.AdamW(p, lr=0.1), I8.AdamW(q2, lr=0.1)
    scale = torch.tensor([1.0], device=DEV)

    def one(o):
        norm, f, bad = o.grad_norm(0.01, grad_scale=scale)
        o.step(grad_scale=f, found_inf=bad)
        return norm
    one(opt), one(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = I8.GradNormPlan([x.grad for x in p]).norm(0.01, grad_scale=scale)
    for i in range(3):
        for a, b, x in zip(p, q2, grads([5000, 300], "bf16", 5 + i)):
            a.grad.copy_(x)
            b.grad.copy_(x)
        scale.fill_(0.5 + i)
        graph.replay()
        eager = I8.GradNormPlan([x.grad for x in q2]).norm(0.01, grad_scale=scale)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(norm, eager))
