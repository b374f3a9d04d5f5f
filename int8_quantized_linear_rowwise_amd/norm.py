"""Layer norm and its gradient: binding of int8_layer_norm_forward /
int8_layer_norm_backward (include/int8lin.h), autograd function and module."""
from __future__ import annotations

from typing import Optional

import torch

from ._lib import check, lib
from ._tensors import _check_out, _code, _empty, _gpu, _on_gpu, _ptr, _raw_stream, _workspace


def _weights(X, weight, bias):
    C = X.shape[1]
    if weight.shape != (C,) or weight.dtype not in (X.dtype, torch.float32):
        raise ValueError(f"weight must have shape ({C},) and X's dtype or float32")
    if bias is not None and (bias.shape != (C,) or bias.dtype != weight.dtype):
        raise ValueError(f"bias must have shape ({C},) and weight's dtype")


def layer_norm_forward(X: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                       out: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
                       rstd: Optional[torch.Tensor] = None):
    """(out, mean, rstd): layer norm of the rows of X (T x C) in X's dtype; mean and rstd fp32, one value a row.

    weight, bias: C values of X's dtype or fp32. out may be X."""
    if X.dim() != 2:
        raise ValueError("X must be 2-D (flatten leading dimensions)")
    T, C = X.shape
    _weights(X, weight, bias)
    _check_out(out, (T, C), X.dtype, "out")
    _check_out(mean, (T,), torch.float32, "mean")
    _check_out(rstd, (T,), torch.float32, "rstd")
    dev = _gpu(X, "X")
    if out is None:
        out = torch.empty_like(X, memory_format=torch.contiguous_format)
    if mean is None:
        mean = _empty((T,), torch.float32, X.device)
    if rstd is None:
        rstd = torch.empty_like(mean)
    with _on_gpu(dev):
        check(lib.int8_layer_norm_forward(_ptr(X, "X", dev), _code(X), T, C, _ptr(weight, "weight", dev),
                                          _ptr(bias, "bias", dev), _code(weight), eps, _ptr(out, "out", dev),
                                          _ptr(mean, "mean", dev), _ptr(rstd, "rstd", dev), _raw_stream(dev)),
              "int8_layer_norm_forward")
    return out, mean, rstd


def layer_norm_backward(G: torch.Tensor, X: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: torch.Tensor, with_grad_X: bool = True, with_grad_weight: bool = True,
                        with_grad_bias: bool = True, grad_X: Optional[torch.Tensor] = None,
                        grad_weight: Optional[torch.Tensor] = None, grad_bias: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None):
    """(grad_X, grad_weight, grad_bias) of layer_norm_forward, None where not asked for; the weight's and the
    bias's gradients in weight's dtype. grad_X may be G when neither of those is asked for."""
    if X.dim() != 2 or G.shape != X.shape or G.dtype != X.dtype:
        raise ValueError("G and X must be 2-D with the same shape and dtype")
    T, C = X.shape
    _weights(X, weight, None)
    if mean.shape != (T,) or rstd.shape != (T,) or mean.dtype != torch.float32 or rstd.dtype != torch.float32:
        raise ValueError(f"mean and rstd must be float32 of shape ({T},)")
    _check_out(grad_X, (T, C), X.dtype, "grad_X")
    _check_out(grad_weight, (C,), weight.dtype, "grad_weight")
    _check_out(grad_bias, (C,), weight.dtype, "grad_bias")
    dev = _gpu(G, "G")
    if grad_X is None and with_grad_X:
        grad_X = torch.empty_like(X, memory_format=torch.contiguous_format)
    if grad_weight is None and with_grad_weight:
        grad_weight = torch.empty_like(weight, memory_format=torch.contiguous_format)
    if grad_bias is None and with_grad_bias:
        grad_bias = torch.empty_like(weight, memory_format=torch.contiguous_format)
    ws = _workspace(workspace, lib.int8_layer_norm_backward_workspace_bytes(T, C), X.device, dev)
    with _on_gpu(dev):
        check(lib.int8_layer_norm_backward(_ptr(G, "G", dev), _ptr(X, "X", dev), _code(X), T, C,
                                           _ptr(mean, "mean", dev), _ptr(rstd, "rstd", dev),
                                           _ptr(weight, "weight", dev), _code(weight),
                                           _ptr(grad_X, "grad_X", dev), _ptr(grad_weight, "grad_weight", dev),
                                           _ptr(grad_bias, "grad_bias", dev), _ptr(ws, "workspace", dev),
                                           0 if ws is None else ws.numel(), _raw_stream(dev)),
              "int8_layer_norm_backward")
    return grad_X, grad_weight, grad_bias


class LayerNormFunction(torch.autograd.Function):
    """Layer norm over the last dimension."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        X = x.reshape(-1, x.shape[-1]).contiguous()
        out, mean, rstd = layer_norm_forward(X, weight.contiguous(), bias, eps)
        ctx.save_for_backward(X, mean, rstd, weight)
        ctx.has_bias = bias is not None
        return out.reshape(x.shape)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        X, mean, rstd, weight = ctx.saved_tensors
        need = ctx.needs_input_grad
        gX, gw, gb = layer_norm_backward(g.reshape(X.shape).contiguous(), X, mean, rstd, weight.contiguous(),
                                         with_grad_X=need[0], with_grad_weight=need[1],
                                         with_grad_bias=ctx.has_bias and need[2])
        return gX.reshape(g.shape) if need[0] else None, gw, gb, None


class LayerNorm(torch.nn.Module):
    """Layer norm over the last dimension with a trainable weight and bias (the input's dtype or fp32)."""

    def __init__(self, features: int, eps: float = 1e-5, bias: bool = True, device=None,
                 dtype: torch.dtype = torch.float32):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(features, device=device, dtype=dtype)) if bias else None
        self.eps = float(eps)

    def forward(self, x):
        return LayerNormFunction.apply(x, self.weight, self.bias, self.eps)
