"""The experts' entry points and the gradient norm refuse bad arguments on the host, before any HIP call (nothing here
touches a GPU); the plain 64-bit forms that the GPU tests use are checked against torch and against differences."""
import ctypes
import math

import pytest
import torch

from tests import _experts as X
from tests.test_abi import FAKE, L  # noqa: F401  (fixture: builds the library if it is missing)


def caller(f, base):
    def call(**kw):
        a = dict(base, **kw)
        return f(*(a[k] for k in base))
    return call


def test_sort_host_errors(L):  # noqa: F811
    need = L.lib.int8_expert_sort_workspace_bytes
    call = caller(L.lib.int8_expert_sort, dict(ids=FAKE, b=8, T=9000, k=2, E=8, off=FAKE, tok=FAKE, pos=FAKE, ws=FAKE,
                                               wsb=1 << 30, st=None))
    assert call(b=2) == L.I8L_EDTYPE
    for k in ("T", "k", "E"):
        assert call(**{k: -1}) == L.I8L_EINVAL, k
    for k in ("ids", "off", "tok", "pos"):
        assert call(**{k: 0}) == L.I8L_EINVAL, k
    assert call(E=L.I8L_SORT_MAX_EXPERTS + 1) == L.I8L_ESHAPE
    assert call(T=(1 << 24) + 1, k=1) == L.I8L_ESHAPE and call(T=1 << 23, k=3) == L.I8L_ESHAPE
    assert call(T=1 << 40, k=1 << 40) == L.I8L_ESHAPE
    wsb = need(9000, 2, 8)
    assert wsb > 0 and wsb % 256 == 0 and need(1, 2, 8) == 0 and need(-1, 2, 8) == 0
    assert call(wsb=wsb - 1) == L.I8L_EWORKSPACE and call(ws=0) == L.I8L_EWORKSPACE
    assert call(ws=FAKE + 4) == L.I8L_EINVAL


def test_forward_host_errors(L):  # noqa: F811
    need = L.lib.int8_expert_forward_workspace_bytes
    call = caller(L.lib.int8_expert_forward,
                  dict(X=FAKE, dt=2, T=8, K=64, rows=FAKE, R=16, CB=FAKE, SCB=FAKE, E=4, N=32, off=FAKE, ids=None, S=4,
                       tau=6.0, out=FAKE, ws=FAKE, wsb=1 << 40, st=None))
    assert call(dt=3) == L.I8L_EDTYPE and call(dt=-1) == L.I8L_EDTYPE
    for k in ("T", "K", "R", "E", "N", "S"):
        assert call(**{k: -1}) == L.I8L_EINVAL, k
    for k in ("X", "CB", "SCB", "off", "out"):
        assert call(**{k: 0}) == L.I8L_EINVAL, k
    assert call(rows=0) == L.I8L_EINVAL                       # without indices there are as many rows as tokens
    assert call(K=L.I8L_MAX_K + 1) == L.I8L_ESHAPE and call(N=L.I8L_MAX_COLS + 1) == L.I8L_ESHAPE
    assert call(R=(1 << 24) + 1) == L.I8L_ESHAPE and call(T=(1 << 24) + 1) == L.I8L_ESHAPE
    assert call(S=65537) == L.I8L_ESHAPE and call(E=65537) == L.I8L_ESHAPE
    assert call(E=65536, N=65536) == L.I8L_ESHAPE             # more scales than an int counts
    wsb = need(8, 64, FAKE, 16, 32, 4)
    assert wsb > 0 and wsb % 256 == 0
    assert need(-1, 64, FAKE, 16, 32, 4) == 0 and need(8, L.I8L_MAX_K + 1, FAKE, 16, 32, 4) == 0
    assert need(4, 64, FAKE, 8, 32, 4) == 0                   # up to four tokens are quantized on the way
    assert need(4, 72, FAKE, 8, 32, 4) == 0                   # any contraction of whole words
    assert need(4, 64, FAKE + 1, 8, 32, 4) > 0 and need(4, 70, FAKE, 8, 32, 4) > 0 and need(4, 64, FAKE, 999, 32, 4) > 0
    assert call(wsb=wsb - 1) == L.I8L_EWORKSPACE and call(ws=0) == L.I8L_EWORKSPACE
    assert call(ws=FAKE + 16) == L.I8L_EINVAL
    assert call(R=0, out=0) == L.I8L_OK and call(N=0, out=0, CB=0, SCB=0) == L.I8L_OK


def test_backward_host_errors(L):  # noqa: F811
    call = caller(L.lib.int8_expert_backward, dict(G=FAKE, dt=1, R=16, N=32, CB=FAKE, SCB=FAKE, E=4, K=64, off=FAKE,
                                                   ids=None, S=4, gX=FAKE, ws=None, wsb=0, st=None))
    assert call(dt=7) == L.I8L_EDTYPE
    for k in ("R", "N", "E", "K", "S"):
        assert call(**{k: -1}) == L.I8L_EINVAL, k
    for k in ("G", "CB", "SCB", "off", "gX"):
        assert call(**{k: 0}) == L.I8L_EINVAL, k
    assert call(R=(1 << 24) + 1) == L.I8L_ESHAPE and call(S=65537) == L.I8L_ESHAPE
    assert call(R=0, G=0, gX=0) == L.I8L_OK and call(K=0, gX=0, CB=0) == L.I8L_OK
    need = L.lib.int8_expert_backward_workspace_bytes
    assert need(FAKE, 1, 16, 32) == 0 and need(FAKE + 2, 1, 16, 32) == 1024
    assert need(FAKE, 2, 16, 33) == 1280 and need(FAKE, 0, 16, 32) == 1024
    assert need(FAKE, 1, -1, 32) == 0 and need(FAKE, 5, 16, 32) == 0
    for bad in (dict(dt=0), dict(N=33, dt=2), dict(G=FAKE + 2)):
        assert call(**bad) == L.I8L_EWORKSPACE and call(**bad, ws=FAKE, wsb=1023) == L.I8L_EWORKSPACE
        assert call(**bad, ws=FAKE + 16, wsb=1 << 20) == L.I8L_EINVAL


def test_combine_host_errors(L):  # noqa: F811
    call = caller(L.lib.int8_expert_combine, dict(Y=FAKE, dt=0, R=16, N=32, pos=FAKE, gate=FAKE, base=None, T=8, k=2,
                                                  out=FAKE, st=None))
    assert call(dt=3) == L.I8L_EDTYPE
    for k in ("R", "N", "T", "k"):
        assert call(**{k: -1}) == L.I8L_EINVAL, k
    for k in ("Y", "pos", "out"):
        assert call(**{k: 0}) == L.I8L_EINVAL, k
    assert call(k=65) == L.I8L_ESHAPE and call(N=L.I8L_MAX_COLS + 1) == L.I8L_ESHAPE
    assert call(T=(1 << 24) + 1) == L.I8L_ESHAPE
    assert call(T=0, out=0) == L.I8L_OK and call(N=0, out=0) == L.I8L_OK
    call = caller(L.lib.int8_expert_combine_backward, dict(G=FAKE, dt=0, T=8, N=32, pos=FAKE, gate=FAKE, k=2, Y=FAKE,
                                                           R=16, n=None, gY=FAKE, gg=FAKE, st=None))
    assert call(dt=-2) == L.I8L_EDTYPE
    for k in ("R", "N", "T", "k"):
        assert call(**{k: -1}) == L.I8L_EINVAL, k
    for k in ("G", "pos", "Y"):
        assert call(**{k: 0}) == L.I8L_EINVAL, k
    assert call(k=65) == L.I8L_ESHAPE and call(R=(1 << 24) + 1) == L.I8L_ESHAPE
    assert call(gY=0, gg=0) == L.I8L_OK


def test_grad_norm_host_errors(L):  # noqa: F811
    f, need = L.lib.int8_grad_norm, L.lib.int8_grad_norm_workspace_bytes

    def table(*rows):
        return (L.GradTensor * len(rows))(*[L.GradTensor(g, n, dt, 0) for g, n, dt in rows])

    def call(t, count=None, kind=2, top=1.0, norm=FAKE, factor=FAKE, bad=FAKE, ws=FAKE, wsb=1 << 30):
        return f(t, len(t) if count is None else count, kind, top, None, 0, norm, factor, bad, ws, wsb, None)
    ok = table((FAKE, 1 << 20, 2), (FAKE, 5, 0))
    assert call(ok, count=-1) == L.I8L_EINVAL and call(ok, count=(1 << 24) + 1) == L.I8L_ESHAPE
    assert call(ok, kind=1) == L.I8L_EINVAL
    assert call(ok, top=-1.0) == L.I8L_EINVAL and call(ok, top=math.nan) == L.I8L_EINVAL
    for k in ("norm", "factor", "bad"):
        assert call(ok, **{k: 0}) == L.I8L_EINVAL, k
    assert need(ok, 2) == 1280 and need(ok, -1) == 0           # 129 partial sums
    assert need(table((FAKE, 100, 2)), 1) == 0 and need(table((FAKE, 1 << 17, 2)), 1) == 0
    assert need(table((FAKE, (1 << 17) + 1, 2)), 1) == 256 and need(table(*[(FAKE, 1, 0)] * 17), 17) == 256
    assert call(ok, wsb=129 * 8 - 1) == L.I8L_EWORKSPACE and call(ok, ws=0) == L.I8L_EWORKSPACE
    assert call(ok, ws=FAKE + 8) == L.I8L_EINVAL
    assert call(table((FAKE, 100, 3))) == L.I8L_EDTYPE
    assert call(table((FAKE, -1, 2))) == L.I8L_EINVAL and call(table((0, 1, 2))) == L.I8L_EINVAL
    assert call(table((FAKE + 1, 1, 2))) == L.I8L_EINVAL and call(table((FAKE + 2, 1, 0))) == L.I8L_EINVAL
    assert call(table((FAKE, (1 << 40) + 1, 2))) == L.I8L_ESHAPE
    assert call(table(*[(FAKE, 1 << 40, 2)] * 5)) == L.I8L_ESHAPE
    assert ctypes.sizeof(L.GradTensor) == 24


def test_bindings_refuse(L):  # noqa: F811
    """What the Python layer checks before it asks for a GPU."""
    import int8_quantized_linear_rowwise_amd as I8
    x, off, pos = torch.zeros(4, 8), torch.zeros(3, dtype=torch.int32), torch.zeros((4, 2), dtype=torch.int32)
    CB, SCB = torch.zeros((2, 6, 8), dtype=torch.int8), torch.zeros((2, 6))
    bad = [
        lambda: I8.expert_sort(torch.zeros(4, dtype=torch.int64), 2),
        lambda: I8.expert_sort(torch.zeros((4, 2)), 2),
        lambda: I8.expert_sort(torch.zeros((4, 2), dtype=torch.int64), 1025),
        lambda: I8.expert_sort(torch.zeros((4, 2), dtype=torch.int64), 2, seg_offsets=off[:2]),
        lambda: I8.expert_sort(torch.zeros((4, 2), dtype=torch.int64), 2),        # not on a GPU
        lambda: I8.expert_forward(x[0], CB, SCB, off),
        lambda: I8.expert_forward(x, CB[0], SCB, off),
        lambda: I8.expert_forward(x, CB, SCB.double(), off),
        lambda: I8.expert_forward(x[:, :4], CB, SCB, off),
        lambda: I8.expert_forward(x, CB, SCB, off.long()),
        lambda: I8.expert_forward(x, CB, SCB, off, seg_expert=off),
        lambda: I8.expert_forward(x, CB, SCB, off, rows=pos),
        lambda: I8.expert_forward(x, CB, SCB, off, out=torch.zeros(5, 6)),
        lambda: I8.expert_forward(x, CB, SCB, off),
        lambda: I8.expert_backward(x, CB, SCB, off),
        lambda: I8.expert_backward(x[:, :6], CB, SCB, off, grad_X=torch.zeros(4, 7)),
        lambda: I8.expert_combine(x, pos.long()),
        lambda: I8.expert_combine(x, pos, gate=torch.zeros(4, 3)),
        lambda: I8.expert_combine(x, pos, gate=torch.zeros((4, 2), dtype=torch.float64)),
        lambda: I8.expert_combine(x, pos, base=torch.zeros(5, 8)),
        lambda: I8.expert_combine_backward(x, pos, with_grad_gate=True),
        lambda: I8.expert_combine_backward(x[:3], pos, with_grad_gate=False),
        lambda: I8.expert_combine_backward(x, pos, Y=x.half()),
        lambda: I8.expert_combine_backward(x, pos, Y=x, n_rows=off),
        lambda: I8.GradNormPlan([]),
        lambda: I8.GradNormPlan([x]),
        lambda: I8.Int8Experts(x),
        lambda: I8.clip_grad_norm_([], -1.0),
        lambda: I8.clip_grad_norm_([], 1.0, norm_type=1.0),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    assert float(I8.clip_grad_norm_([x], 1.0)) == 0.0


# ---- the plain forms ------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("T,k,E,drop", [(1, 1, 1, 0), (7, 2, 5, 0.3), (40, 4, 9, 0.1), (0, 2, 3, 0)])
def test_plain_sort(T, k, E, drop):
    ids = X.choices(T, k, E, 3, drop)
    off, token, position = X.sort(ids, E)
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True).indices
    n = int((flat >= 0).sum())
    assert off.tolist() == [int(((flat >= 0) & (flat < e)).sum()) for e in range(E + 1)]
    assert torch.equal(token[:n].long(), (order // k)[:n]) and (token[n:] == -1).all()
    for i in range(T * k):
        p = int(position.view(-1)[i])
        assert (p == -1) == (int(flat[i]) < 0) and (p < 0 or int(order[p]) == i)


def test_plain_forward_against_oracle():
    """One expert is the projection itself."""
    import numpy as np
    import oracle
    CB, SCB = X.weights(1, 20, 50, 1)
    x = X.inputs(9, 50, "f32", 2)
    y, _ = X.forward(x, CB, SCB, torch.tensor([0, 9]))
    f = oracle.linear_forward(x.numpy(), "f32", CB[0].numpy(), SCB[0].numpy(), None, 6.0)
    np.testing.assert_allclose(y.numpy(), f["y"], rtol=1e-12, atol=1e-12)
    G = X.inputs(9, 20, "f32", 3, 0)
    g, _ = X.backward(G, CB, SCB, torch.tensor([0, 9]))
    b = oracle.linear_backward_input(G.numpy(), "f32", CB[0].numpy(), SCB[0].numpy())
    np.testing.assert_allclose(g.numpy(), b["y"], rtol=1e-12, atol=1e-12)


def test_plain_forward_rows_and_segments():
    CB, SCB = X.weights(3, 11, 24, 1)
    x = X.inputs(6, 24, "f16", 2)
    rows = torch.tensor([5, 0, 0, 9, -1, 2, 1], dtype=torch.int32)
    y, _ = X.forward(x, CB, SCB, torch.tensor([0, 2, 5, 6]), torch.tensor([2, 0, 7]), rows)
    for r, (e, t) in enumerate([(2, 5), (2, 0), (0, 0), (None, 0), (None, 0), (None, 0), (None, 0)]):
        if e is None:
            assert (y[r] == 0).all()
        else:
            alone, _ = X.forward(x, CB[e:e + 1], SCB[e:e + 1], torch.tensor([0, 6]))
            assert torch.equal(y[r], alone[t])


def test_plain_combine_gradient_against_differences():
    pos = torch.tensor([[0, 3], [2, -1], [9, 1]], dtype=torch.int32)
    g = torch.Generator().manual_seed(1)
    Y, gate, base, G = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((5, 4), (3, 2), (3, 4), (3, 4)))
    gY, gg, _ = X.combine_backward(G, pos, gate, Y, 5)
    h = 1e-6

    def loss(Y, gate):
        return float((X.combine(Y, pos, gate, base)[0] * G).sum())
    for a, ga in ((Y, gY), (gate, gg)):
        for i in range(a.numel()):
            b = a.clone().view(-1)
            b[i] += h
            up = loss(*((b.view_as(a), gate) if a is Y else (Y, b.view_as(a))))
            b[i] -= 2 * h
            dn = loss(*((b.view_as(a), gate) if a is Y else (Y, b.view_as(a))))
            # a second difference of a bilinear form is 0: what is left is cancellation, 2^-52 |loss| / h
            assert abs((up - dn) / (2 * h) - float(ga.view(-1)[i])) < 1e-8


def test_plain_norm_against_torch():
    g = [torch.randn(n) for n in (5, 0, 17)]
    p = [torch.nn.Parameter(torch.zeros_like(x)) for x in g]
    for kind in (2, math.inf):
        norm, factor = X.grad_norm(g, 0.5, kind)
        for q, x in zip(p, g):
            q.grad = x.clone()
        ref = torch.nn.utils.clip_grad_norm_([q for q in p if q.numel()], 0.5, kind)
        assert abs(float(ref) - norm) < 1e-5 * norm
        assert torch.allclose(p[0].grad, g[0] * factor, rtol=1e-5)
