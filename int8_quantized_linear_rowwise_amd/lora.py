"""Low-rank adapters of many requests beside the frozen int8 projection.

The token rows lie in consecutive segments (requests when serving, sequences
when training); each segment uses one adapter of a stack, or none. Binding of
int8_lora_forward / int8_lora_backward (include/int8lin.h), the autograd
function that joins them to the int8 layer, and a module.
"""
from __future__ import annotations

from typing import Optional

import torch

from ._lib import I8L_LORA_MAX_RANK, check, lib
from ._tensors import _check_out, _code, _empty, _gpu, _on_gpu, _ptr, _raw_stream, _workspace


def _segments(seg_offsets, seg_adapter):
    """Number of segments; one segment of all rows without offsets."""
    if seg_offsets is None:
        n = 1
    else:
        if seg_offsets.dim() != 1 or seg_offsets.numel() < 1 or seg_offsets.dtype != torch.int32:
            raise ValueError("seg_offsets must be a 1-D int32 tensor of (number of segments + 1) row offsets")
        n = seg_offsets.numel() - 1
    if seg_adapter is not None and (seg_adapter.dtype != torch.int32 or seg_adapter.shape != (n,)):
        raise ValueError(f"seg_adapter must be int32 with one entry for each of the {n} segments")
    return n


def _adapters(A, B, scaling, dtype, K, N):
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError("A must be (adapters, rank, K) and B (adapters, N, rank)")
    n, R = A.shape[:2]
    if A.shape[2] != K or B.shape != (n, N, R) or A.dtype != dtype or B.dtype != dtype:
        raise ValueError(f"A must be {dtype} (adapters, rank, {K}) and B {dtype} (adapters, {N}, rank), "
                         f"got {A.dtype} {tuple(A.shape)} and {B.dtype} {tuple(B.shape)}")
    if scaling.shape != (n,) or scaling.dtype != torch.float32:
        raise ValueError("scaling must be float32 with one factor for each adapter")
    return n, R


def lora_forward(X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scaling: torch.Tensor,
                 seg_offsets: Optional[torch.Tensor] = None, seg_adapter: Optional[torch.Tensor] = None,
                 base: Optional[torch.Tensor] = None, with_v: bool = False, out: Optional[torch.Tensor] = None,
                 v: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """out[t] = base[t] + scaling[a] * B[a] (A[a] x[t]) for the adapter a of row t's segment, in X's dtype.

    X: T x K; A: adapters x R x K and B: adapters x N x R (X's dtype); scaling:
    adapters fp32. seg_offsets: int32, segments + 1 row offsets from 0 to T (None:
    one segment); seg_adapter: int32, each segment's adapter, any value outside
    [0, adapters) for none (None: segment j uses adapter j). base: T x N or None
    for 0; out may be base. with_v: also return V = A[a] x[t] (T x R fp32), which
    lora_backward needs."""
    if X.dim() != 2:
        raise ValueError("X must be 2-D (flatten leading dimensions)")
    T, K = X.shape
    N = B.shape[1] if B.dim() == 3 else -1
    n, R = _adapters(A, B, scaling, X.dtype, K, N)
    S = _segments(seg_offsets, seg_adapter)
    if base is not None:
        _check_out(base, (T, N), X.dtype, "base")
    if out is not None:
        _check_out(out, (T, N), X.dtype, "out")
    if v is not None:
        _check_out(v, (T, R), torch.float32, "v")
    dev = _gpu(X, "X")
    if out is None:
        out = _empty((T, N), X.dtype, X.device) if base is None else \
            torch.empty_like(base, memory_format=torch.contiguous_format)
    if v is None and with_v:
        v = _empty((T, R), torch.float32, X.device)
    need = lib.int8_lora_forward_workspace_bytes(T, K, N, R, S)
    ws = _workspace(workspace, need, X.device, dev)
    with _on_gpu(dev):
        check(lib.int8_lora_forward(_ptr(X, "X", dev), _code(X), T, K, _ptr(A, "A", dev), _ptr(B, "B", dev),
                                    _ptr(scaling, "scaling", dev), n, R, N, _ptr(seg_offsets, "seg_offsets", dev),
                                    _ptr(seg_adapter, "seg_adapter", dev), S, _ptr(base, "base", dev),
                                    _ptr(out, "out", dev), _ptr(v, "v", dev), _ptr(ws, "workspace", dev),
                                    0 if ws is None else ws.numel(), _raw_stream(dev)),
              "int8_lora_forward")
    return (out, v) if with_v else out


def lora_backward(G: torch.Tensor, X: torch.Tensor, V: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                  scaling: torch.Tensor, seg_offsets: Optional[torch.Tensor] = None,
                  seg_adapter: Optional[torch.Tensor] = None, base_grad: Optional[torch.Tensor] = None,
                  with_grad_X: bool = True, with_grad_A: bool = True, with_grad_B: bool = True,
                  grad_X: Optional[torch.Tensor] = None, grad_A: Optional[torch.Tensor] = None,
                  grad_B: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Gradients of lora_forward: (grad_X, grad_A, grad_B), None where not asked for.

    G: T x N; V: the forward's T x R fp32; base_grad: T x K added to grad_X (the
    projection's own input gradient) or None; grad_X may be base_grad. An adapter
    without rows gets a zero gradient."""
    if G.dim() != 2 or X.dim() != 2 or G.shape[0] != X.shape[0] or G.dtype != X.dtype:
        raise ValueError("G (T x N) and X (T x K) must be 2-D with the same number of rows and dtype")
    T, N = G.shape
    K = X.shape[1]
    n, R = _adapters(A, B, scaling, X.dtype, K, N)
    S = _segments(seg_offsets, seg_adapter)
    if V.shape != (T, R) or V.dtype != torch.float32:
        raise ValueError(f"V must be float32 of shape {(T, R)}")
    _check_out(base_grad, (T, K), X.dtype, "base_grad")
    _check_out(grad_X, (T, K), X.dtype, "grad_X")
    _check_out(grad_A, A.shape, X.dtype, "grad_A")
    _check_out(grad_B, B.shape, X.dtype, "grad_B")
    dev = _gpu(G, "G")
    if grad_X is None and with_grad_X:
        grad_X = torch.empty_like(X, memory_format=torch.contiguous_format)
    if grad_A is None and with_grad_A:
        grad_A = torch.empty_like(A, memory_format=torch.contiguous_format)
    if grad_B is None and with_grad_B:
        grad_B = torch.empty_like(B, memory_format=torch.contiguous_format)
    need = lib.int8_lora_backward_workspace_bytes(T, K, N, R, n, S)
    ws = _workspace(workspace, need, X.device, dev)
    with _on_gpu(dev):
        check(lib.int8_lora_backward(_ptr(G, "G", dev), _ptr(X, "X", dev), _ptr(V, "V", dev), _code(X), T, K,
                                     _ptr(A, "A", dev), _ptr(B, "B", dev), _ptr(scaling, "scaling", dev), n, R, N,
                                     _ptr(seg_offsets, "seg_offsets", dev), _ptr(seg_adapter, "seg_adapter", dev), S,
                                     _ptr(base_grad, "base_grad", dev), _ptr(grad_X, "grad_X", dev),
                                     _ptr(grad_A, "grad_A", dev), _ptr(grad_B, "grad_B", dev),
                                     _ptr(ws, "workspace", dev), 0 if ws is None else ws.numel(), _raw_stream(dev)),
              "int8_lora_backward")
    return grad_X, grad_A, grad_B


class Int8LoraFunction(torch.autograd.Function):
    """The frozen int8 layer with adapters beside it: forward in int8 plus the
    adapters' product, backward through the memory-efficient kernel plus the
    adapters' gradients. The int8 weight is frozen, and scaling is constant."""

    @staticmethod
    def forward(ctx, x, CB, SCB, bias, A, B, scaling, seg_offsets, seg_adapter, threshold):
        from . import int8_linear_forward
        X = x.reshape(-1, x.shape[-1]).contiguous()
        out = int8_linear_forward(X, CB, SCB, bias, threshold)
        out, V = lora_forward(X, A, B, scaling, seg_offsets, seg_adapter, base=out, out=out, with_v=True)
        ctx.save_for_backward(X, V, CB, SCB, A, B, scaling, seg_offsets, seg_adapter)
        ctx.shape = x.shape
        ctx.has_bias = bias is not None
        return out.reshape(*x.shape[:-1], CB.shape[0])

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        from . import int8_linear_backward_input
        X, V, CB, SCB, A, B, scaling, seg_offsets, seg_adapter = ctx.saved_tensors
        need = ctx.needs_input_grad
        if need[6]:   # forward cannot tell this from a call under no_grad, which is fine
            raise ValueError("scaling has no gradient here: the adapters' factors are constants (detach it)")
        g2 = g.reshape(-1, g.shape[-1]).contiguous()
        need_b = ctx.has_bias and need[3]
        gX = gb = None
        if need[0] or need_b:
            gX, gb = int8_linear_backward_input(g2, CB, SCB, with_grad_bias=need_b)
        _, gA, gB = lora_backward(g2, X, V, A, B, scaling, seg_offsets, seg_adapter,
                                  base_grad=gX if need[0] else None, grad_X=gX if need[0] else None,
                                  with_grad_X=need[0], with_grad_A=need[4], with_grad_B=need[5])
        return gX.reshape(ctx.shape) if need[0] else None, None, None, gb, gA, gB, None, None, None, None


class Int8LoraLinear(torch.nn.Module):
    """Frozen int8 linear layer with `adapters` trainable low-rank adapters of one rank beside it.

    A is drawn uniformly with variance 1 / (3 K), B is zero, so a new adapter
    changes nothing; each adapter's product is multiplied by alpha / rank."""

    def __init__(self, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, adapters: int = 1, rank: int = 16,
                 alpha: float = 16.0, threshold: float = 6.0, dtype: Optional[torch.dtype] = None):
        super().__init__()
        from . import quantize_weight
        if not 1 <= rank <= I8L_LORA_MAX_RANK:
            raise ValueError(f"rank must be 1 to {I8L_LORA_MAX_RANK}")
        N, K = weight.shape
        dtype = weight.dtype if dtype is None else dtype
        CB, SCB = quantize_weight(weight.detach().contiguous())
        self.register_buffer("CB", CB)
        self.register_buffer("SCB", SCB)
        self.register_buffer("scaling", torch.full((adapters,), alpha / rank, device=weight.device))
        self.bias = torch.nn.Parameter(bias.detach().clone()) if bias is not None else None
        self.lora_A = torch.nn.Parameter(
            torch.empty((adapters, rank, K), device=weight.device).uniform_(-K ** -0.5, K ** -0.5).to(dtype))
        self.lora_B = torch.nn.Parameter(torch.zeros((adapters, N, rank), dtype=dtype, device=weight.device))
        self.threshold = float(threshold)

    def forward(self, x, seg_offsets=None, seg_adapter=None):
        """x: (..., K); its rows (leading dimensions flattened) lie in segments as lora_forward takes them.
        Without segments all rows use adapter 0."""
        b = self.bias.to(x.dtype) if self.bias is not None else None
        return Int8LoraFunction.apply(x, self.CB, self.SCB, b, self.lora_A.to(x.dtype), self.lora_B.to(x.dtype),
                                      self.scaling, seg_offsets, seg_adapter, self.threshold)
