"""Norm of all gradients, and clipping by it: binding of int8_grad_norm
(include/int8lin.h). What it returns is what AdamW's step takes: the factor as
grad_scale, so that clipping costs no pass of its own, and found_inf."""
from __future__ import annotations

import ctypes
import math
from typing import Iterable, Optional, Sequence, Tuple

import torch

from ._lib import I8L_F32, I8L_NORM_INF, GradTensor, check, lib
from ._tensors import DTYPE_CODE, _empty, _on_gpu, _ptr, _raw_stream, _workspace


def _numbers(max_norm: Optional[float], norm_type: float) -> Tuple[float, int]:
    max_norm = math.inf if max_norm is None else float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError(f"max_norm must be a number of 0 or more, got {max_norm}")
    if norm_type not in (2, math.inf):
        raise ValueError(f"norm_type must be 2 or infinity, got {norm_type}")
    return max_norm, 2 if norm_type == 2 else I8L_NORM_INF


class GradNormPlan:
    """The gradients of a step, checked once; `norm` and `clip` read (and write) the memory that these tensors have now
    at every call, and the plan keeps it alive: a gradient that is replaced, or given other memory (g.data = ...), needs
    a new plan, and one whose storage is resized leaves this one without. A captured call's plan is kept as long as the
    graph. Nothing of it lies on the device: every call has outputs and workspace of its own, so calls on different
    streams, or captured into different graphs, do not meet.

    grads: contiguous tensors on one GPU, each fp32, fp16 or bf16."""

    def __init__(self, grads: Sequence[torch.Tensor]):
        grads = list(grads)
        if not grads:
            raise ValueError("no gradients")
        self.device, self.gpu = grads[0].device, grads[0].get_device()
        if self.gpu < 0:
            raise ValueError("gradients must be on a GPU")
        self.count = len(grads)
        rows = []
        for g in grads:
            code = DTYPE_CODE.get(g.dtype)
            if code is None:
                raise TypeError(f"unsupported dtype {g.dtype}; expected float32, float16 or bfloat16")
            rows += (_ptr(g, "every gradient", self.gpu), g.numel(), code)
        self._keep = grads, [g.untyped_storage() for g in grads]
        # i8l_grad_tensor is three 64-bit words, the dtype in the last one's lower half
        self._table = (ctypes.c_int64 * len(rows))(*rows)
        self._overlap: Optional[bool] = None      # found out by the first clipping
        assert ctypes.sizeof(GradTensor) == 24
        self.workspace_bytes = lib.int8_grad_norm_workspace_bytes(self._table, self.count)

    def __reduce__(self):
        """A copy is laid out for the copied gradients, not for the addresses of these."""
        return GradNormPlan, (list(self._keep[0]),)

    def _overlapping(self) -> bool:
        t, end = self._table, 0
        for p, n, code in sorted(zip(t[::3], t[1::3], t[2::3])):
            if n:
                if p < end:
                    return True
                end = p + n * (4 if code == I8L_F32 else 2)
        return False

    def _run(self, max_norm, norm_type, grad_scale, clip, workspace):
        max_norm, kind = _numbers(max_norm, norm_type)
        scale = 0
        if grad_scale is not None:
            if grad_scale.dtype != torch.float32 or grad_scale.numel() != 1 or grad_scale.get_device() != self.gpu:
                raise ValueError(f"grad_scale must be one float32 value on {self.device}")
            scale = grad_scale.data_ptr()
        if clip:
            if self._overlap is None:
                self._overlap = self._overlapping()
            if self._overlap:
                raise ValueError("gradients that overlap, or are in the list twice, would be clipped twice")
        out = _empty((3,), torch.float32, self.device)
        ws = _workspace(workspace, self.workspace_bytes, self.device, self.gpu)
        at = out.data_ptr()
        with _on_gpu(self.gpu):
            check(lib.int8_grad_norm(self._table, self.count, kind, max_norm, scale, clip, at, at + 4, at + 8,
                                     _ptr(ws, "workspace", self.gpu), 0 if ws is None else ws.numel(),
                                     _raw_stream(self.gpu)),
                  "int8_grad_norm")
        return out.unbind()

    def norm(self, max_norm: Optional[float] = None, norm_type: float = 2.0,
             grad_scale: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
        """(norm, factor, found_inf), one fp32 value each: the norm (2, or infinity: the largest magnitude) of all
        gradients times grad_scale; grad_scale * min(1, max_norm / (norm + 1e-6)), what the gradients are to be
        multiplied with (AdamW's grad_scale); and 1 where the norm is not finite, else 0. max_norm None: no clipping."""
        return self._run(max_norm, norm_type, grad_scale, 0, workspace)

    def clip(self, max_norm: Optional[float] = None, norm_type: float = 2.0,
             grad_scale: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
        """`norm`, and the gradients multiplied by the factor in place. No two of them may overlap."""
        return self._run(max_norm, norm_type, grad_scale, 1, workspace)


def clip_grad_norm_(parameters: Iterable[torch.Tensor], max_norm: float, norm_type: float = 2.0,
                    grad_scale: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Clips the gradients of `parameters` (those that have one) in place to a norm of max_norm over all of them, after
    multiplying them by grad_scale if there is one; returns their norm before the clipping. The list is laid out at every
    call (0.3 ms of host time for 448 tensors, a kept GradNormPlan's clip 0.05). It keeps nothing: where the
    call is captured, the gradients and grad_scale are kept by the caller as long as the graph."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    grads = [p.grad for p in parameters if p.grad is not None]
    _numbers(max_norm, norm_type)
    if not grads:
        return torch.tensor(0.0)
    return GradNormPlan(grads).clip(max_norm, norm_type, grad_scale)[0]
