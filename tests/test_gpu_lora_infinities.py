"""Infinities in the adapters' operands: they reach the outputs that the formulas say, and no others. With 16-bit
operands an infinity meets both parts of V or dV, whose second may be 0 or of the other sign, so it can arrive as a
NaN."""
import pytest
import torch

from tests import _finetune as F
from tests.test_gpu_lora import DTS, I8, KEYS, gpu  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu
T, K, N, R, n = 70, 136, 200, 16, 2
SEGS = ([0, 30, 33, 70], [0, -1, 1])


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("what", ["X", "G", "A", "B", "base", "base_grad"])
def test_infinities_arrive_where_the_formulas_say(I8, dt, what):  # noqa: F811
    c = F.lora_inputs(dt, T, K, N, R, n, 12)
    at = {"X": (40, 5), "G": (50, 7), "A": (1, 3, 9), "B": (1, 11, 2), "base": (35, 4), "base_grad": (36, 4)}[what]
    off, ids = (gpu(x) for x in SEGS)

    def calls(c):
        d = {k: gpu(c[k]) for k in KEYS}
        out, V = I8.lora_forward(d["X"], d["A"], d["B"], d["scaling"], off, ids, base=d["base"], with_v=True)
        return (out, V) + I8.lora_backward(d["G"], d["X"], V, d["A"], d["B"], d["scaling"], off, ids,
                                           base_grad=d["base_grad"])

    def formulas(c):
        segs = F.segments_of(*SEGS, n, T)
        y, _, v, _ = F.lora_forward64(c, dt, segs)
        return (y, v) + tuple(w for w, _ in F.lora_backward64(c, dt, segs))

    clean = calls(c)
    c[what][at] = float("inf")
    bad = calls(c)
    torch.cuda.synchronize()
    reached = 0
    for name, a, b, w in zip(("out", "V", "grad_X", "grad_A", "grad_B"), bad, clean, formulas(c)):
        fin = torch.isfinite(w)
        reached += int((~fin).sum())
        assert not torch.isfinite(a.cpu()[~fin]).any(), name
        # a sum in another order would be fine too; these have the same
        assert torch.equal(a.cpu()[fin], b.cpu()[fin]), name
        if dt == "f32" or what.startswith("base"):
            assert torch.equal(a.cpu()[~fin].double(), w[~fin]) or torch.isnan(w[~fin]).any(), name
    assert reached
