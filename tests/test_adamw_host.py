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
