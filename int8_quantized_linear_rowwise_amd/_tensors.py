"""What the bindings share: dtype codes, device pointers and result checks."""
from __future__ import annotations

import contextlib
from typing import Optional

import torch

from ._lib import I8L_BF16, I8L_F16, I8L_F32

DTYPE_CODE = {torch.float32: I8L_F32, torch.float16: I8L_F16, torch.bfloat16: I8L_BF16}


def _code(t: torch.Tensor) -> int:
    try:
        return DTYPE_CODE[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}; expected float32, float16 or bfloat16") from None


def _dev(t: Optional[torch.Tensor], name: str) -> int:
    if t is None:
        return 0
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() if t.numel() > 0 else 0


def _check_out(t: Optional[torch.Tensor], shape: tuple, dtype: torch.dtype, name: str) -> None:
    """Caller-provided result tensors must have exactly the size the kernels write."""
    if t is not None and (t.shape != shape or t.dtype != dtype):
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _empty(shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device)


def _raw_stream(dev: int) -> int:
    """The current HIP stream of GPU number `dev` (torch.cuda.current_stream builds a Stream object first, 2 us)."""
    return torch._C._cuda_getCurrentRawStream(dev)


_HERE = contextlib.nullcontext()


def _on_gpu(dev: int):
    """Makes GPU number `dev` the current one (-1: none): a kernel is launched on the current GPU, whatever GPU its
    stream and its tensors belong to, and the default stream's handle is the same on all of them. (0.25 us where it
    is current already; torch.cuda.current_device asks for the runtime's start first, 0.12 us more.)"""
    return _HERE if dev < 0 or dev == torch._C._cuda_getDevice() else torch.cuda.device(dev)


def _gpu(t: torch.Tensor, name: str) -> int:
    """The number of the GPU that a call's first tensor is on."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    return dev


def _ptr(t: Optional[torch.Tensor], name: str, dev: int) -> int:
    """Device pointer of a tensor that has to be contiguous and on GPU number `dev`; 0 for None."""
    if t is None:
        return 0
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on GPU {dev}, as the call's first tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _workspace(ws: Optional[torch.Tensor], need: int, device, dev: int) -> Optional[torch.Tensor]:
    """The caller's uint8 workspace if there is one, else a new one (None when nothing is needed)."""
    if ws is None:
        return _empty((need,), torch.uint8, device) if need else None
    if ws.dtype != torch.uint8 or ws.numel() < need or ws.get_device() != dev:
        raise ValueError(f"workspace must be uint8 on GPU {dev} with at least {need} bytes")
    return ws
