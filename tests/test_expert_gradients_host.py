"""Positions of any kind in the weighted sum's gradient: what is refused on the host, and the plain form against
differences."""
import pytest
import torch

from tests import _experts as X
from tests._stub_gpu import stub  # noqa: F401  (fixture)
from tests.test_abi import FAKE, L  # noqa: F401  (fixture: builds the library if it is missing)


def test_any_positions_host_errors(L):  # noqa: F811
    base = dict(G=FAKE, dt=L.I8L_ANY_POSITIONS, T=8, N=32, pos=FAKE, gate=FAKE, k=2, Y=FAKE, R=16, n=FAKE, gY=FAKE,
                gg=FAKE, st=None)

    def call(**kw):
        return L.lib.int8_expert_combine_backward(*dict(base, **kw).values())
    assert call(n=0) == L.I8L_EINVAL and call(n=FAKE + 2) == L.I8L_EINVAL           # the scratch
    assert call(dt=L.I8L_ANY_POSITIONS + 3) == L.I8L_EDTYPE and call(dt=L.I8L_ANY_POSITIONS * 2) == L.I8L_EDTYPE
    assert call(dt=-1) == L.I8L_EDTYPE and call(dt=-L.I8L_ANY_POSITIONS) == L.I8L_EDTYPE
    assert call(k=65) == L.I8L_ESHAPE and call(G=0) == L.I8L_EINVAL and call(pos=0) == L.I8L_EINVAL
    assert call(n=0, gY=0, gg=0) == L.I8L_OK


def test_any_positions_bindings(stub, L, monkeypatch):  # noqa: F811
    calls = []
    monkeypatch.setattr(L.lib, "int8_expert_combine_backward", lambda *a: calls.append(a) or 0)
    f = stub.I8.expert_combine_backward
    G, pos = torch.zeros(8, 32), torch.zeros((8, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="n_rows"):
        f(G, pos, with_grad_gate=False, n_rows=torch.zeros(1, dtype=torch.int32), any_positions=True)
    with pytest.raises(ValueError, match="workspace"):
        f(G, pos, with_grad_gate=False, any_positions=True, workspace=torch.zeros(127, dtype=torch.uint8))
    ws = torch.zeros(128, dtype=torch.uint8)
    f(G, pos, with_grad_gate=False, any_positions=True, workspace=ws)
    assert calls[-1][1] == L.I8L_ANY_POSITIONS and calls[-1][9] == ws.data_ptr()
    f(G, pos, Y=torch.zeros(16, 32), with_grad_Y=False, any_positions=True)
    assert calls[-1][9] == 0
    f(G, pos, with_grad_gate=False)
    assert calls[-1][1] == L.I8L_F32 and calls[-1][9] == 0


def test_plain_gradient_of_repeats_against_differences():
    pos = torch.tensor([[0, 0, 3], [3, -1, 1], [9, 3, 0]], dtype=torch.int32)
    g = torch.Generator().manual_seed(1)
    Y, gate, base, G = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((5, 4), (3, 3), (3, 4), (3, 4)))
    gY, _ = X.combine_gradient(G, pos, gate, 5)
    assert (gY[2] == 0).all() and (gY[4] == 0).all()
    h = 1e-6
    for i in range(Y.numel()):
        sides = []
        for sign in (1, -1):
            b = Y.clone()
            b.view(-1)[i] += sign * h
            sides.append(float((X.combine(b, pos, gate, base)[0] * G).sum()))
        # linear in Y: what is left is cancellation, 2^-52 |loss| / h
        assert abs((sides[0] - sides[1]) / (2 * h) - float(gY.view(-1)[i])) < 1e-8


@pytest.mark.parametrize("k,sums", [(1, 1), (64, 1), (65, 2), (150, 3)])
def test_token_gradient_takes_any_number_of_choices(stub, L, monkeypatch, k, sums):  # noqa: F811
    calls = []
    for name in ("int8_expert_forward", "int8_expert_backward", "int8_expert_combine"):
        monkeypatch.setattr(L.lib, name, lambda *a, n=name: calls.append((n, a)) or 0)
    x = torch.zeros((8, 32), dtype=torch.bfloat16, requires_grad=True)
    CB, SCB = torch.zeros((2, 16, 32), dtype=torch.int8), torch.zeros((2, 16))
    off, rows = torch.zeros(3, dtype=torch.int32), torch.zeros(8 * k, dtype=torch.int32)
    pos = torch.zeros((8, k), dtype=torch.int32)
    stub.I8.Int8ExpertsFunction.apply(x, CB, SCB, off, None, rows, pos, 6.0).sum().backward()
    assert [n for n, _ in calls] == ["int8_expert_forward", "int8_expert_backward"] + ["int8_expert_combine"] * sums
    took = [a[8] for n, a in calls if n == "int8_expert_combine"]
    assert sum(took) == k and max(took) <= 64 and x.grad.dtype == x.dtype


def test_token_gradient_takes_positions_of_any_layout(stub, L, monkeypatch):  # noqa: F811
    """A slice of the positions, which the forward takes, is no reason to refuse the gradient."""
    for name in ("int8_expert_forward", "int8_expert_backward", "int8_expert_combine"):
        monkeypatch.setattr(L.lib, name, lambda *a: 0)
    x = torch.zeros((8, 32), requires_grad=True)
    CB, SCB = torch.zeros((2, 16, 32), dtype=torch.int8), torch.zeros((2, 16))
    off, rows = torch.zeros(3, dtype=torch.int32), torch.zeros(16, dtype=torch.int32)
    for pos in (torch.zeros((8, 4), dtype=torch.int32)[:, ::2], torch.zeros((2, 8), dtype=torch.int32).t()):
        stub.I8.Int8ExpertsFunction.apply(x, CB, SCB, off, None, rows, pos, 6.0).sum().backward()
