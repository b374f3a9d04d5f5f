"""What the AdamW optimizer does on the host, with a library that records its calls instead of a GPU."""
import gc
import io
import weakref
from copy import deepcopy

import pytest
import torch

from tests._stub_gpu import L, stub  # noqa: F401  (fixtures)


def params(*sizes):
    P = [torch.nn.Parameter(torch.ones(n)) for n in sizes]
    for p in P:
        p.grad = torch.ones_like(p)
    return P


def test_a_capture_on_the_parameters_gpu_is_seen(stub):  # noqa: F811
    """The gradients of a captured step are held while its graph can be replayed, also where another GPU is current."""
    (p,) = P = params(300)
    opt = stub.I8.AdamW(P)
    opt.step()
    stub.capturing = True
    opt.step()
    gone = weakref.ref(p.grad)
    p.grad = None
    gc.collect()
    assert gone() is not None
    del opt
    gc.collect()
    assert gone() is None


def test_a_captured_step_holds_its_scalars(stub):  # noqa: F811
    """A graph's replays read grad_scale and found_inf: they live as long as the optimizer, those of eager steps only
    as long as their caller keeps them."""
    opt = stub.I8.AdamW(params(300))
    for capturing in (False, True):
        stub.capturing = capturing
        scalars = [torch.ones(1), torch.zeros(1)]
        gone = [weakref.ref(t) for t in scalars]
        opt.step(grad_scale=scalars[0], found_inf=scalars[1])
        stub.args.clear()
        del scalars
        gc.collect()
        assert [r() is None for r in gone] == [not capturing] * 2
    del opt
    gc.collect()
    assert [r() is None for r in gone] == [True] * 2


def test_a_captured_step_holds_its_tensors(stub):  # noqa: F811
    """A replay writes the memory of its capture, also after a parameter or a state got new memory."""
    (p,) = P = params(300)
    opt = stub.I8.AdamW(P)
    opt.step()
    stub.capturing = True
    opt.step()
    stub.capturing = False
    gone = [weakref.ref(t.untyped_storage()) for t in (p, opt.state[p]["m"], opt.state[p]["v"])]
    p.data = torch.zeros(300)
    opt.state[p]["m"] = torch.zeros(300)
    opt.load_state_dict(opt.state_dict())
    gc.collect()
    assert [r() is None for r in gone] == [False] * 3


@pytest.mark.parametrize("what", ["layout", "type", "grad_scale", "found_inf", "lr", "betas", "eps", "weight_decay"])
@pytest.mark.parametrize("before", [0, 2])
def test_a_refused_step_changes_nothing(stub, what, before):  # noqa: F811
    """Everything is checked before the first launch: no group is stepped, no step counted, no state made."""
    a, b = torch.nn.Parameter(torch.ones(4, 6)), torch.nn.Parameter(torch.ones(6, 4).to(torch.bfloat16))
    for p in (a, b):
        p.grad = torch.ones_like(p)
    opt = stub.I8.AdamW([dict(params=[a]), dict(params=[b])], master=True)
    for _ in range(before):
        opt.step()
    launched, made = len(stub.seen), {p: dict(opt.state[p]) for p in opt.state}
    kw, good = {}, b.grad
    if what == "layout":
        b.grad = torch.ones(4, 6).to(torch.bfloat16).t()
    elif what == "type":
        b.grad, b.grad_dtype = None, torch.float32
        b.grad = torch.ones(6, 4)
    elif what in ("grad_scale", "found_inf"):
        kw[what] = torch.ones(1, dtype=torch.float64)
    else:
        was = opt.param_groups[1][what]
        opt.param_groups[1][what] = (0.9, 1.0) if what == "betas" else float("inf")
    for _ in range(2):
        with pytest.raises(ValueError):
            opt.step(**kw)
    assert len(stub.seen) == launched and {p: dict(s) for p, s in opt.state.items()} == made
    b.grad, b.grad_dtype = None, b.dtype
    b.grad = good
    if what in opt.defaults:
        opt.param_groups[1][what] = was
    opt.step()
    assert len(stub.seen) == launched + 2
    assert [x[8] for x in stub.args[-2:]] == [opt.state[p]["step"] for p in (a, b)] == [before + 1] * 2


@pytest.mark.parametrize("how", ["deepcopy", "saved"])
def test_a_copy_steps_on_its_own(stub, how):  # noqa: F811
    """A copied optimizer lays out a plan of its own tensors: nothing that it launches names the original's."""
    opt = stub.I8.AdamW(params(300, 40), state_bits=8)
    opt.step()
    own = opt._plans
    if how == "deepcopy":
        copy = deepcopy(opt)
    else:
        file = io.BytesIO()
        torch.save(opt, file)
        file.seek(0)
        copy = torch.load(file, weights_only=False)
    for p in copy.param_groups[0]["params"]:
        p.grad = torch.ones_like(p)
    copy.step()
    assert opt._plans is own and stub.args[-1][0] != stub.args[0][0]
    assert [s["step"] for s in copy.state.values()] == [2, 2] and [s["step"] for s in opt.state.values()] == [1, 1]
    for s in copy.state.values():
        assert s["m"].dtype == torch.float8_e4m3fn and s["m_scale"].dtype == torch.float32


@pytest.mark.parametrize("kw", [dict(lr=-1.0), dict(lr=float("nan")), dict(betas=(2, 0.9)), dict(betas=(0.9, 1.0)),
                                dict(betas=(0.9,)), dict(eps=-1e-8), dict(weight_decay=-0.1),
                                dict(weight_decay=float("inf")), dict(state_bits=16)])
def test_numbers_out_of_range_are_refused_at_once(stub, kw):  # noqa: F811
    """By the constructor, for its defaults and for a group's own numbers, and by add_param_group."""
    (p, q) = params(3, 4)
    with pytest.raises(ValueError):
        stub.I8.AdamW([p], **kw)
    with pytest.raises(ValueError):
        stub.I8.AdamW([dict(params=[p], **kw)])
    opt = stub.I8.AdamW([p])
    with pytest.raises(ValueError):
        opt.add_param_group(dict(params=[q], **kw))
    opt.step()
    assert len(opt.param_groups) == 1 and len(stub.seen) == 1


@pytest.mark.parametrize("what", ["first step", "other gradients"])
def test_a_capture_of_a_step_without_its_plan_is_refused(stub, what):  # noqa: F811
    """Making states (their zeros would be written at every replay) and copying a plan to the GPU do not belong in a
    graph: one ordinary step with the same gradients comes first. The refused step leaves nothing behind."""
    (p,) = P = params(300)
    opt = stub.I8.AdamW(P)
    done = 0
    if what == "other gradients":
        opt.step()
        p.grad, done = torch.ones(300), 1
    stub.capturing = True
    with pytest.raises(RuntimeError, match="before the capture"):
        opt.step()
    assert len(stub.seen) == done and len(opt.state) == done and not opt._captured
    with pytest.raises(RuntimeError, match="before the capture"):
        stub.I8.AdamWPlan([p.detach()], [p.grad], [torch.zeros(300)], [torch.zeros(300)])
    stub.capturing = False
    opt.step()
    stub.capturing = True
    opt.step()
    assert opt.state[p]["step"] == done + 2 and len(opt._captured) == 1


def test_parameters_off_the_gpu_are_refused(L):  # noqa: F811
    import int8_quantized_linear_rowwise_amd as I8
    opt = I8.AdamW(params(30))
    with pytest.raises(ValueError, match="GPU"):
        opt.step()
    assert not opt.state
