"""What the AdamW optimizer does on the host, with a library that records its calls instead of a GPU."""
import gc
import weakref

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
