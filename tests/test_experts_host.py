"""What the experts' bindings and the gradient norm do on the host, with a library that records its calls instead of a
GPU: the GPU a call launches on, workspaces, what a captured call holds, and gradients that are not asked for."""
import gc
import weakref

import pytest
import torch

from tests._stub_gpu import L, stub  # noqa: F401  (fixtures)

ENTRIES = ["int8_expert_sort", "int8_expert_forward", "int8_expert_backward", "int8_expert_combine",
           "int8_expert_combine_backward", "int8_grad_norm"]


@pytest.fixture
def lib(stub, L, monkeypatch):  # noqa: F811
    def entry(name):
        def call(*a):
            stub.seen.append((name, stub.current))
            stub.args.append(a)
            return 0
        return call
    for name in ENTRIES:
        monkeypatch.setattr(L.lib, name, entry(name))
    return stub


def sizes():
    x = torch.zeros(8, 32, dtype=torch.float16)
    CB, SCB = torch.zeros((2, 16, 32), dtype=torch.int8), torch.zeros((2, 16))
    return x, CB, SCB, torch.zeros(3, dtype=torch.int32), torch.zeros((8, 2), dtype=torch.int32)


def test_every_entry_point_runs_on_its_tensors_gpu(lib):
    I8 = lib.I8
    x, CB, SCB, off, pos = sizes()
    off2, token, pos2 = I8.expert_sort(pos, 2)
    assert off2.shape == (3,) and token.shape == (16,) and pos2.shape == (8, 2)
    y = I8.expert_forward(x, CB, SCB, off, rows=token)
    assert y.shape == (16, 16) and I8.expert_backward(y, CB, SCB, off).shape == (16, 32)
    gate = torch.zeros(8, 2)
    out = I8.expert_combine(y, pos, gate)
    gY, gg = I8.expert_combine_backward(out, pos, gate, y, n_rows=off[-1:])
    assert gY.shape == y.shape and gg.shape == gate.shape
    plan = I8.GradNormPlan([x, gate])
    assert all(v.shape == () for v in plan.norm(1.0)) and len(plan.clip(1.0)) == 3
    assert {n for n, _ in lib.seen} == set(ENTRIES)
    assert {d for _, d in lib.seen} == {1} and lib.current == 0


def test_calls_have_workspaces_of_their_own(lib):
    """Nothing on the device is shared between two calls of one plan, which may run at once."""
    I8 = lib.I8
    plan = I8.GradNormPlan([torch.zeros(1 << 20)])
    kept = [plan.norm(1.0), plan.norm(1.0)]
    a, b = lib.args[-2:]
    assert len({a[6], b[6], a[9], b[9]}) >= 3 and a[6] != b[6]
    assert kept[0][0].data_ptr() == a[6] and kept[1][2].data_ptr() == b[8]


def test_a_captured_norm_holds_the_gradients_and_the_scale(lib):
    P = [torch.nn.Parameter(torch.ones(300))]
    P[0].grad = torch.ones(300)
    opt = lib.I8.AdamW(P)
    opt.step()
    for capturing in (False, True):
        lib.capturing = capturing
        scale = torch.ones(1)
        opt.grad_norm(1.0, grad_scale=scale)
        gone = weakref.ref(scale)
        del scale
        gc.collect()
        assert (gone() is not None) == capturing
    grad = weakref.ref(P[0].grad)
    P[0].grad = None
    gc.collect()
    assert grad() is not None
    del opt
    gc.collect()
    assert grad() is None and gone() is None


def test_clip_takes_generators_single_tensors_and_parameters_without_gradients(lib):
    I8 = lib.I8
    p = [torch.nn.Parameter(torch.ones(n)) for n in (3, 4, 5)]
    p[0].grad, p[2].grad = torch.ones(3), torch.ones(5)
    I8.clip_grad_norm_((q for q in p), 1.0)
    assert lib.args[-1][1] == 2 and lib.args[-1][5] == 1
    I8.clip_grad_norm_(p[0], 1.0, float("inf"))
    assert lib.args[-1][1] == 1 and lib.args[-1][2] == 0
    calls = len(lib.seen)
    assert float(I8.clip_grad_norm_([p[1]], 1.0)) == 0.0 and len(lib.seen) == calls


def test_gradients_that_are_not_asked_for_are_not_computed(lib):
    I8 = lib.I8
    x, CB, SCB, off, pos = sizes()
    Y, gate, base = torch.zeros(16, 16), torch.zeros(8, 2), torch.zeros((8, 16), requires_grad=True)
    I8.ExpertCombineFunction.apply(Y, pos, gate, base, off[-1:]).sum().backward()
    assert [n for n, _ in lib.seen] == ["int8_expert_combine"] and (base.grad == 1).all()
    I8.ExpertCombineFunction.apply(Y, pos, gate.requires_grad_(), None, off[-1:]).sum().backward()
    assert lib.seen[-1][0] == "int8_expert_combine_backward" and lib.args[-1][10] == 0 and lib.args[-1][11] != 0
    I8.ExpertCombineFunction.apply(Y.requires_grad_(), pos, gate.detach(), None, off[-1:]).sum().backward()
    assert lib.args[-1][10] != 0 and lib.args[-1][11] == 0 and lib.args[-1][7] == 0      # Y is not kept, nor read
    lib.seen.clear()
    m = I8.Int8ExpertsFunction.apply(x, CB, SCB, off, None, None, None, 6.0)
    assert not m.requires_grad
    I8.Int8ExpertsFunction.apply(x.requires_grad_(), CB, SCB, off, None, None, None, 6.0).sum().backward()
    assert [n for n, _ in lib.seen] == ["int8_expert_forward"] * 2 + ["int8_expert_backward"]


def test_refused_calls_leave_the_current_gpu(lib, monkeypatch):
    from int8_quantized_linear_rowwise_amd import _lib
    I8 = lib.I8
    x, CB, SCB, off, pos = sizes()
    for name, call in (("int8_expert_sort", lambda: I8.expert_sort(pos, 2)),
                       ("int8_expert_forward", lambda: I8.expert_forward(x, CB, SCB, off)),
                       ("int8_grad_norm", lambda: I8.GradNormPlan([x]).norm())):
        monkeypatch.setattr(_lib.lib, name, lambda *a: _lib.I8L_ESHAPE)
        with pytest.raises(I8.Int8LinError):
            call()
        assert lib.current == 0
