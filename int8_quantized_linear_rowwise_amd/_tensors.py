"""What the bindings share: dtype codes, device pointers and result checks."""
from __future__ import annotations

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
    if t is not None and (tuple(t.shape) != tuple(shape) or t.dtype != dtype):
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _empty(shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device)


def _same_device(first: torch.Tensor, **others: Optional[torch.Tensor]) -> None:
    """The kernels run on `first`'s GPU: every other tensor has to be there too."""
    for name, t in others.items():
        if t is not None and t.device != first.device:
            raise ValueError(f"{name} is on {t.device}, expected {first.device}")


def _workspace(ws: Optional[torch.Tensor], need: int, device) -> Optional[torch.Tensor]:
    """The caller's uint8 workspace if there is one, else a new one (None when nothing is needed)."""
    if ws is None:
        return _empty((need,), torch.uint8, device) if need else None
    if ws.dtype != torch.uint8 or ws.numel() < need or ws.device != device:
        raise ValueError(f"workspace must be uint8 on {device} with at least {need} bytes")
    return ws
