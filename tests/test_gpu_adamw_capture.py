"""Captured AdamW steps on the GPU: replays after the caller has dropped what the capture named, and a capture that is
refused."""
import gc

import pytest
import torch

from tests.test_gpu_adamw import I8  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def pair(I8, bits):  # noqa: F811
    g = torch.Generator().manual_seed(3)
    p, q = (torch.nn.Parameter(torch.ones(3000, device="cuda:0")) for _ in range(2))
    p.grad = torch.randn(3000, generator=g).cuda()
    q.grad = p.grad.clone()
    return p, q, I8.AdamW([p], state_bits=bits), I8.AdamW([q], state_bits=bits)


@pytest.mark.parametrize("bits", [32, 8])
def test_replays_after_the_scalars_are_dropped(I8, bits):  # noqa: F811
    p, q, ours, ref = pair(I8, bits)
    scale, inf = torch.tensor([0.25], device="cuda:0"), torch.zeros(1, device="cuda:0")
    keep = scale.clone(), inf.clone()
    ours.step(grad_scale=scale, found_inf=inf)
    ref.step(grad_scale=keep[0], found_inf=keep[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ours.step(grad_scale=scale, found_inf=inf)
    del scale, inf
    gc.collect()
    for _ in range(3):
        junk = [torch.full((1,), 3.0, device="cuda:0") for _ in range(64)]
        torch.cuda.synchronize()
        graph.replay()
        ref.state[q]["step"] = 1
        ref.step(grad_scale=keep[0], found_inf=keep[1])
        torch.cuda.synchronize()
        assert torch.equal(p, q)
        del junk


@pytest.mark.parametrize("bits", [32, 8])
def test_a_refused_capture_leaves_everything_as_it_was(I8, bits):  # noqa: F811
    p, q, ours, ref = pair(I8, bits)
    x = torch.zeros(8, device="cuda:0")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.add_(1)
        with pytest.raises(RuntimeError, match="before the capture"):
            ours.step()
    for number in (1, 2):
        graph.replay()
        ours.step()
        ref.step()
        torch.cuda.synchronize()
        assert torch.equal(p, q) and ours.state[p]["step"] == number and (x == number).all()
