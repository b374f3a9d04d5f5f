"""CPU tensors that say they are on GPU 1 while GPU 0 is current, and a library
that records which GPU is current when an entry point is called: what the
bindings do on the host, shown without a GPU."""
import pytest
import torch

from tests.test_abi import L  # noqa: F401  (fixture: builds the library if it is missing)

ENTRIES = ["int8_quantize_rowwise", "int8_linear_forward", "int8_linear_forward_noalloc", "int8_linear_forward_flagged",
           "int8_linear_forward_check", "int8_silu_outlier_flags", "int8_linear_backward_input",
           "int8_linear_backward_input_int8", "int8_linear_backward_weight", "int8_lora_forward", "int8_lora_backward",
           "int8_layer_norm_forward", "int8_layer_norm_backward", "int8_adamw_step"]


class Stub:
    def __init__(self, I8):
        self.I8 = I8
        self.current = 0          # the current GPU
        self.seen = []            # (entry point, the GPU that was current)
        self.args = []            # its arguments
        self.capturing = False


@pytest.fixture
def stub(L, monkeypatch):  # noqa: F811
    import int8_quantized_linear_rowwise_amd as I8
    s = Stub(I8)

    class Device:
        def __init__(self, i):
            self.i = i if isinstance(i, int) else 1

        def __enter__(self):
            self.before, s.current = s.current, self.i

        def __exit__(self, *e):
            s.current = self.before

    class Stream:
        cuda_stream = 0

    def entry(name):
        def call(*a):
            s.seen.append((name, s.current))
            s.args.append(a)
            return 0
        return call

    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: s.current, raising=False)
    # a stream of GPU 1 is captured, if any
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: s.capturing and s.current == 1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    for name in ENTRIES:
        monkeypatch.setattr(L.lib, name, entry(name))
    return s
