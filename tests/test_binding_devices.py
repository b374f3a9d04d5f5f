"""Kernels are launched on the current GPU, whatever stream and tensors a call
names: every binding makes its tensors' GPU the current one for the call. Shown
on the CPU with tensors that say they are on GPU 1 while GPU 0 is current, and
a library that records which GPU is current when it is called."""
import pytest
import torch

from tests.test_abi import L  # noqa: F401  (fixture: builds the library if it is missing)

ENTRIES = ["int8_quantize_rowwise", "int8_linear_forward", "int8_linear_forward_noalloc", "int8_linear_forward_flagged",
           "int8_linear_forward_check", "int8_silu_outlier_flags", "int8_linear_backward_input",
           "int8_linear_backward_input_int8", "int8_linear_backward_weight", "int8_lora_forward", "int8_lora_backward",
           "int8_layer_norm_forward", "int8_layer_norm_backward", "int8_adamw_step"]


@pytest.fixture
def calls(L, monkeypatch):  # noqa: F811
    import int8_quantized_linear_rowwise_amd as I8
    current, seen = [0], []

    class Device:
        def __init__(self, i):
            self.i = i if isinstance(i, int) else i.index

        def __enter__(self):
            self.before, current[0] = current[0], self.i

        def __exit__(self, *e):
            current[0] = self.before

    class Stream:
        cuda_stream = 0

    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    for name in ENTRIES:
        monkeypatch.setattr(L.lib, name, lambda *a, n=name: seen.append((n, current[0])) or 0)
    return I8, seen, current


def test_every_entry_point_runs_on_its_tensors_gpu(calls):
    I8, seen, current = calls
    h, f = torch.float16, torch.float32
    X, G, bias = torch.zeros(4, 16, dtype=h), torch.zeros(4, 6, dtype=h), torch.zeros(6, dtype=h)
    CB, SCB = torch.zeros(6, 16, dtype=torch.int8), torch.ones(6)
    CBt, SCBt = torch.zeros(16, 6, dtype=torch.int8), torch.ones(16)
    I8.int8_quantize_rowwise(X)
    I8.int8_linear_forward(X, CB, SCB, bias)
    I8.int8_linear_forward_noalloc(X, CB, SCB, bias)
    flags = I8.outlier_flags_buffer(4, 16, "cpu")
    I8.silu_outlier_flags(X, flags=flags)
    I8.int8_linear_forward_flagged(X, flags, CB, SCB, bias)
    I8.forward_check(I8.forward_workspace(4, 16, 6, 16, "cpu"), 4, 16, 6, 16)
    I8.int8_linear_backward_input(G, CB, SCB)
    I8.int8_linear_backward_input_int8(G, CBt, SCBt)
    I8.int8_linear_backward_weight(G, X)
    A, B, s = torch.zeros(2, 8, 16, dtype=h), torch.zeros(2, 6, 8, dtype=h), torch.ones(2)
    off = torch.tensor([0, 1, 4], dtype=torch.int32)
    _, V = I8.lora_forward(X, A, B, s, off, with_v=True)
    I8.lora_backward(G, X, V, A, B, s, off)
    w = torch.ones(16, dtype=h)
    _, mean, rstd = I8.layer_norm_forward(X, w)
    I8.layer_norm_backward(X, X, mean, rstd, w)
    I8.AdamWPlan([w], [w.clone()], [torch.zeros(16, dtype=f)], [torch.zeros(16, dtype=f)]).step(1, 1e-3)
    assert sorted({n for n, _ in seen}) == sorted(ENTRIES)
    assert {d for _, d in seen} == {1}, [n for n, d in seen if d != 1]
    assert current == [0]


def test_the_current_gpu_stays_when_a_call_is_refused(calls, monkeypatch):
    I8, _, current = calls
    from int8_quantized_linear_rowwise_amd import _lib
    monkeypatch.setattr(_lib.lib, "int8_layer_norm_forward", lambda *a: _lib.I8L_EINVAL)
    with pytest.raises(I8.Int8LinError):
        I8.layer_norm_forward(torch.zeros(4, 16), torch.ones(16))
    assert current == [0]
