"""Kernels are launched on the current GPU, whatever stream and tensors a call
names: every binding makes its tensors' GPU the current one for the call."""
import pytest
import torch

from tests._stub_gpu import ENTRIES, L, stub  # noqa: F401  (fixtures)


def test_every_entry_point_runs_on_its_tensors_gpu(stub):  # noqa: F811
    I8 = stub.I8
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
    assert sorted({n for n, _ in stub.seen}) == sorted(ENTRIES)
    assert {d for _, d in stub.seen} == {1}, [n for n, d in stub.seen if d != 1]
    assert stub.current == 0


def test_the_current_gpu_stays_when_a_call_is_refused(stub, monkeypatch):  # noqa: F811
    I8 = stub.I8
    from int8_quantized_linear_rowwise_amd import _lib
    monkeypatch.setattr(_lib.lib, "int8_layer_norm_forward", lambda *a: _lib.I8L_EINVAL)
    with pytest.raises(I8.Int8LinError):
        I8.layer_norm_forward(torch.zeros(4, 16), torch.ones(16))
    assert stub.current == 0
