"""Clipping on the GPU: factor, flag and every tensor against the 64-bit form, with a scale, with gradients that are not
finite, and as part of a captured step."""
import math

import pytest
import torch

from tests import _experts as X
from tests._gpu import TORCH

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# lists of one launch, of several launches over one list, and of several lists
LISTS = [[1], [0, 5, 0], [131072], [5] * 16, [131073], [5] * 17, [8191, 8192, 8193] * 9, [300] * 281, [4, 16384] * 150]


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


def clipped(a, b, f, factor, dt):
    """a = D(f b), and f within a rounding of the 64-bit factor: a against factor b in 64 bits, with the factor's
    rounding, the product's and the type's."""
    assert torch.equal(a, (b.float() * f).to(b.dtype))
    y = b.to(X.d) * factor
    X.check(a, y, X.rounded(y, 2 * 2.0 ** -24 * y.abs() + 2.0 ** -150, dt), "clipped")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", LISTS)
@pytest.mark.parametrize("kind", [2, math.inf])
@pytest.mark.parametrize("c,part", [(None, 3.0), (0.5, 8.0), (4.0, 2.0), (0.25, 0.5), (-2.0, 3.0)])
def test_clip_against_the_factor(I8, dt, sizes, kind, c, part):
    """part: how many times as large as max_norm the norm is (below 1: only the scale is applied)."""
    g = grads(sizes, dt)
    before = [x.clone() for x in g]
    full, _ = X.grad_norm(g, math.inf, kind, 1.0 if c is None else c)
    want, factor = X.grad_norm(g, full / part, kind, 1.0 if c is None else c)
    scale = None if c is None else torch.tensor([c], device=DEV)
    norm, f, bad = I8.GradNormPlan(g).clip(full / part, kind, scale)
    assert near(norm, want) and near(f, factor) and float(bad) == 0
    assert factor != 1.0
    for a, b in zip(g, before):
        clipped(a, b, f, factor, {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}[b.dtype])


def test_clip_of_unaligned_tensors(I8):
    raw = grads([300001], "f16")[0]
    for a, b in ((1, 40000), (40003, 300001)):
        keep = raw.clone()
        g = [raw[a:b]]
        full, _ = X.grad_norm(g)
        want, factor = X.grad_norm(g, full / 3)
        norm, f, bad = I8.GradNormPlan(g).clip(full / 3)
        assert near(norm, want) and near(f, factor) and float(bad) == 0
        clipped(raw[a:b], keep[a:b], f, factor, "f16")
        assert torch.equal(raw[:a], keep[:a]) and torch.equal(raw[b:], keep[b:])


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("sizes", [[1000, 24], [200000, 24], [700] * 300])
@pytest.mark.parametrize("kind", [2, math.inf])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_clip_of_what_is_not_finite(I8, dt, sizes, kind, value):
    """An infinite norm: the factor 0, which leaves NaN where the infinity was; a norm of NaN: NaN everywhere."""
    g = grads(sizes, dt)
    g[-1][7] = value
    before = [x.clone() for x in g]
    norm, f, bad = I8.GradNormPlan(g).clip(1.0, kind, torch.tensor(0.5, device=DEV))
    assert float(bad) == 1
    assert math.isnan(float(f)) if math.isnan(value) else float(f) == 0 and math.isinf(float(norm))
    for a, b in zip(g, before):
        torch.testing.assert_close(a, (b.float() * f).to(b.dtype), rtol=0, atol=0, equal_nan=True)
    nan = sum(int(a.isnan().sum()) for a in g)
    assert nan == (sum(sizes) if math.isnan(value) else 1)


def test_captured_clip(I8):
    """One graph of a clipping: replays clip what the gradients then hold by the scale that then holds."""
    g = grads([5000, 300, 140000], "bf16")
    plan = I8.GradNormPlan(g)
    scale = torch.ones(1, device=DEV)
    plan.clip(0.05, 2, scale)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        there = plan.clip(0.05, 2, scale)
    for i in range(5):
        new = grads([5000, 300, 140000], "bf16", 10 + i)
        if i == 3:
            new[1][4] = math.inf
        for a, b in zip(g, new):
            a.copy_(b)
        scale.fill_(0.5 + i)
        torch.cuda.synchronize()
        graph.replay()
        here = I8.GradNormPlan(new).clip(0.05, 2, scale)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(there, here)), i
        for a, b in zip(g, new):
            torch.testing.assert_close(a, b, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_norm_and_step(I8, bits):
    """Norm and AdamW step in one graph, factor and flag read at each replay: the same parameters as an optimizer that
    takes the same step eagerly, a step with an infinity left out by both."""
    sizes = [5000, 300, 140000]
    start = grads(sizes, "bf16", 1, 1.0)
    mine, theirs = ([torch.nn.Parameter(x.clone()) for x in start] for _ in range(2))
    for q, r, x in zip(mine, theirs, grads(sizes, "bf16", 2)):
        q.grad, r.grad = x.clone(), x.clone()
    opt, ref = (I8.AdamW(p, lr=0.1, state_bits=bits) for p in (mine, theirs))
    scale = torch.ones(1, device=DEV)

    def one(o):
        norm, f, bad = o.grad_norm(0.05, grad_scale=scale)
        o.step(grad_scale=f, found_inf=bad)
        return norm, f, bad
    one(opt), one(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        there = one(opt)
    for i in range(5):
        new = grads(sizes, "bf16", 10 + i)
        if i == 2:
            new[2][99] = math.inf
        for q, r, x in zip(mine, theirs, new):
            q.grad.copy_(x), r.grad.copy_(x)
        scale.fill_(0.5 + i)
        torch.cuda.synchronize()
        graph.replay()
        before = [r.detach().clone() for r in theirs]
        for r in theirs:                          # a captured step keeps its number, the second
            ref.state[r]["step"] = 1
        here = one(ref)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(there, here)), i
        assert float(here[2]) == (1 if i == 2 else 0)
        for q, r, b in zip(mine, theirs, before):
            assert torch.equal(q, r), i
            assert torch.equal(r, b) == (i == 2), i
            for a, c in zip(opt.state[q].values(), ref.state[r].values()):
                if isinstance(a, torch.Tensor):
                    assert torch.equal(a.view(torch.uint8), c.view(torch.uint8)), i
