"""Experts of a mixture with frozen int8 weights: the sort of tokens by expert,
the products of each expert's rows, and the weighted sum back to tokens.
Binding of int8_expert_* (include/int8lin.h), autograd functions and a module.

    ids, gate = ...                                    # (T, k): each token's experts and their weights
    off, token, position = expert_sort(ids, E)
    h = experts(x, off, rows=token, position=position)     # Int8Experts: (T, K) -> (T k, N), sorted by expert
    y = ExpertCombineFunction.apply(h, position, gate, residual, None)
"""
from __future__ import annotations

from typing import Optional

import torch

from ._lib import I8L_ANY_POSITIONS, I8L_SORT_MAX_EXPERTS, check, lib
from ._tensors import _check_out, _code, _empty, _gpu, _on_gpu, _ptr, _raw_stream, _workspace


def expert_sort(experts: torch.Tensor, n_experts: int, seg_offsets: Optional[torch.Tensor] = None,
                row_token: Optional[torch.Tensor] = None, position: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None):
    """Rows for the choices `experts` (T x k int32 or int64), sorted by expert and, within an expert, by token.

    Returns (seg_offsets: n_experts + 1 int32, the first row of each expert; row_token: T k int32, the token of each
    row, -1 behind the last; position: T x k int32, the row of each choice). A choice outside [0, n_experts) is not
    routed: it has no row, its position is -1."""
    if experts.dim() != 2 or experts.dtype not in (torch.int32, torch.int64):
        raise ValueError("experts must be T x k, int32 or int64")
    if not 0 <= n_experts <= I8L_SORT_MAX_EXPERTS:
        raise ValueError(f"n_experts must be 0 to {I8L_SORT_MAX_EXPERTS}")
    T, k = experts.shape
    dev, device = _gpu(experts, "experts"), experts.device
    _check_out(seg_offsets, (n_experts + 1,), torch.int32, "seg_offsets")
    _check_out(row_token, (T * k,), torch.int32, "row_token")
    _check_out(position, (T, k), torch.int32, "position")
    if seg_offsets is None:
        seg_offsets = _empty((n_experts + 1,), torch.int32, device)
    if row_token is None:
        row_token = _empty((T * k,), torch.int32, device)
    if position is None:
        position = _empty((T, k), torch.int32, device)
    ws = _workspace(workspace, lib.int8_expert_sort_workspace_bytes(T, k, n_experts), device, dev)
    with _on_gpu(dev):
        check(lib.int8_expert_sort(_ptr(experts, "experts", dev), experts.element_size(), T, k, n_experts,
                                   _ptr(seg_offsets, "seg_offsets", dev), _ptr(row_token, "row_token", dev),
                                   _ptr(position, "position", dev), _ptr(ws, "workspace", dev),
                                   0 if ws is None else ws.numel(), _raw_stream(dev)),
              "int8_expert_sort")
    return seg_offsets, row_token, position


def _weights(CB, SCB):
    if CB.dim() != 3 or CB.dtype != torch.int8 or SCB.dtype != torch.float32 or SCB.shape != CB.shape[:2]:
        raise ValueError("CB must be (experts, N, K) int8 and SCB (experts, N) float32")
    return CB.shape


def _segments(seg_offsets, seg_expert):
    if seg_offsets.dim() != 1 or seg_offsets.numel() < 1 or seg_offsets.dtype != torch.int32:
        raise ValueError("seg_offsets must be a 1-D int32 tensor of (number of segments + 1) row offsets")
    n = seg_offsets.numel() - 1
    if seg_expert is not None and (seg_expert.dtype != torch.int32 or seg_expert.shape != (n,)):
        raise ValueError(f"seg_expert must be int32 with one entry for each of the {n} segments")
    return n


def _rows(rows):
    if rows is not None and (rows.dim() != 1 or rows.dtype != torch.int32):
        raise ValueError("rows must be a 1-D int32 tensor of token numbers")


def expert_forward(X: torch.Tensor, CB: torch.Tensor, SCB: torch.Tensor, seg_offsets: torch.Tensor,
                   seg_expert: Optional[torch.Tensor] = None, rows: Optional[torch.Tensor] = None,
                   threshold: float = 6.0, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """out[r] = the int8 product (with outlier columns) of token rows[r] with its row's expert, in X's dtype.

    X: T x K; CB: experts x N x K int8 and SCB: experts x N fp32 (quantize_weight of the experts' rows). seg_offsets:
    int32, segments + 1 row offsets; seg_expert: int32, each segment's expert (None: segment j uses expert j; any value
    outside [0, experts): none). rows: int32, the token of each row, any value outside [0, T) for none (None: row r is
    token r). A row without expert or token, and every row behind the last offset, becomes 0. Tokens that no row names
    (padding) count for the outlier columns too: fill them with finite values."""
    if X.dim() != 2:
        raise ValueError("X must be 2-D (flatten leading dimensions)")
    T, K = X.shape
    E, N, K2 = _weights(CB, SCB)
    if K2 != K:
        raise ValueError(f"CB's rows must have X's {K} features")
    S = _segments(seg_offsets, seg_expert)
    _rows(rows)
    R = T if rows is None else rows.numel()
    _check_out(out, (R, N), X.dtype, "out")
    dev = _gpu(X, "X")
    if out is None:
        out = _empty((R, N), X.dtype, X.device)
    cb = _ptr(CB, "CB", dev)
    ws = _workspace(workspace, lib.int8_expert_forward_workspace_bytes(T, K, cb, R, N, S), X.device, dev)
    with _on_gpu(dev):
        check(lib.int8_expert_forward(_ptr(X, "X", dev), _code(X), T, K, _ptr(rows, "rows", dev), R,
                                      cb, _ptr(SCB, "SCB", dev), E, N,
                                      _ptr(seg_offsets, "seg_offsets", dev), _ptr(seg_expert, "seg_expert", dev), S,
                                      threshold, _ptr(out, "out", dev), _ptr(ws, "workspace", dev),
                                      0 if ws is None else ws.numel(), _raw_stream(dev)),
              "int8_expert_forward")
    return out


def expert_backward(G: torch.Tensor, CB: torch.Tensor, SCB: torch.Tensor, seg_offsets: torch.Tensor,
                    seg_expert: Optional[torch.Tensor] = None, grad_X: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None):
    """grad_X[r] = fp16(G[r]) @ dequant(CB of r's expert), one row for each row of G (R x N), in G's dtype; 0 for rows
    without an expert. The rows of a token are added up by expert_combine without a gate."""
    if G.dim() != 2:
        raise ValueError("G must be 2-D (flatten leading dimensions)")
    R, N = G.shape
    E, N2, K = _weights(CB, SCB)
    if N2 != N:
        raise ValueError(f"CB must have G's {N} output features")
    S = _segments(seg_offsets, seg_expert)
    _check_out(grad_X, (R, K), G.dtype, "grad_X")
    dev = _gpu(G, "G")
    if grad_X is None:
        grad_X = _empty((R, K), G.dtype, G.device)
    g, code = _ptr(G, "G", dev), _code(G)
    ws = _workspace(workspace, lib.int8_expert_backward_workspace_bytes(g, code, R, N), G.device, dev)
    with _on_gpu(dev):
        check(lib.int8_expert_backward(g, code, R, N, _ptr(CB, "CB", dev), _ptr(SCB, "SCB", dev),
                                       E, K, _ptr(seg_offsets, "seg_offsets", dev),
                                       _ptr(seg_expert, "seg_expert", dev), S, _ptr(grad_X, "grad_X", dev),
                                       _ptr(ws, "workspace", dev), 0 if ws is None else ws.numel(),
                                       _raw_stream(dev)),
              "int8_expert_backward")
    return grad_X


def _positions(position, gate):
    if position.dim() != 2 or position.dtype != torch.int32:
        raise ValueError("position must be T x k int32")
    if gate is not None and (gate.shape != position.shape or gate.dtype != torch.float32):
        raise ValueError("gate must be float32 of position's shape")
    return position.shape


def expert_combine(Y: torch.Tensor, position: torch.Tensor, gate: Optional[torch.Tensor] = None,
                   base: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """out[t] = base[t] + sum_j gate[t, j] Y[position[t, j]], in Y's dtype.

    Y: R x N; position: T x k int32, any value outside [0, R) is left out; gate: T x k fp32 or None for 1; base: T x N
    or None for 0; out may be base."""
    if Y.dim() != 2:
        raise ValueError("Y must be 2-D")
    R, N = Y.shape
    T, k = _positions(position, gate)
    _check_out(base, (T, N), Y.dtype, "base")
    _check_out(out, (T, N), Y.dtype, "out")
    dev = _gpu(Y, "Y")
    if out is None:
        out = _empty((T, N), Y.dtype, Y.device)
    with _on_gpu(dev):
        check(lib.int8_expert_combine(_ptr(Y, "Y", dev), _code(Y), R, N, _ptr(position, "position", dev),
                                      _ptr(gate, "gate", dev), _ptr(base, "base", dev), T, k, _ptr(out, "out", dev),
                                      _raw_stream(dev)),
              "int8_expert_combine")
    return out


def expert_combine_backward(G: torch.Tensor, position: torch.Tensor, gate: Optional[torch.Tensor] = None,
                            Y: Optional[torch.Tensor] = None, n_rows: Optional[torch.Tensor] = None,
                            rows: Optional[int] = None, with_grad_Y: bool = True, with_grad_gate: bool = True,
                            grad_Y: Optional[torch.Tensor] = None, grad_gate: Optional[torch.Tensor] = None,
                            any_positions: bool = False, workspace: Optional[torch.Tensor] = None):
    """(grad_Y, grad_gate) of expert_combine, None where not asked for.

    G: T x N. Y, the forward's, is read for grad_gate only; without it `rows` is the number of its rows (default: T k).
    Without any_positions, no two positions may name the same row, and rows of grad_Y that no position names are left
    as they were, in a new grad_Y uninitialised; with n_rows (one int32 on the GPU: the sort's last offset) the rows
    from there on are 0. With any_positions a row that several name gets the sum of their terms, a row that none names
    0, n_rows is not needed, and the workspace takes 8 bytes a row of grad_Y."""
    if G.dim() != 2:
        raise ValueError("G must be 2-D")
    T, k = _positions(position, gate)
    N = G.shape[1]
    if G.shape[0] != T:
        raise ValueError(f"G must have position's {T} rows")
    if Y is not None and (Y.dim() != 2 or Y.shape[1] != N or Y.dtype != G.dtype):
        raise ValueError(f"Y must be {G.dtype} with {N} columns")
    if with_grad_gate and Y is None:
        raise ValueError("the gate's gradient needs Y")
    R = Y.shape[0] if Y is not None else T * k if rows is None else int(rows)
    if n_rows is not None and (n_rows.dtype != torch.int32 or n_rows.numel() != 1):
        raise ValueError("n_rows must be one int32 value")
    if any_positions and n_rows is not None:
        raise ValueError("n_rows says which rows no position names; with any_positions that is found out")
    _check_out(grad_Y, (R, N), G.dtype, "grad_Y")
    _check_out(grad_gate, (T, k), torch.float32, "grad_gate")
    dev = _gpu(G, "G")
    if grad_Y is None and with_grad_Y:
        grad_Y = _empty((R, N), G.dtype, G.device)
    if grad_gate is None and with_grad_gate:
        grad_gate = _empty((T, k), torch.float32, G.device)
    code = _code(G)
    if any_positions:
        code |= I8L_ANY_POSITIONS
        n_rows = _workspace(workspace, 8 * R if with_grad_Y else 0, G.device, dev)
    with _on_gpu(dev):
        check(lib.int8_expert_combine_backward(_ptr(G, "G", dev), code, T, N, _ptr(position, "position", dev),
                                               _ptr(gate, "gate", dev), k, _ptr(Y, "Y", dev), R,
                                               _ptr(n_rows, "workspace" if any_positions else "n_rows", dev),
                                               _ptr(grad_Y, "grad_Y", dev) if with_grad_Y else 0,
                                               _ptr(grad_gate, "grad_gate", dev) if with_grad_gate else 0,
                                               _raw_stream(dev)),
              "int8_expert_combine_backward")
    return grad_Y if with_grad_Y else None, grad_gate if with_grad_gate else None


MAX_CHOICES = 64     # rows of a token that one weighted sum takes


def _sum_of_rows(gX, position):
    """Each token's rows added up; more of them than one sum takes in fp32, rounded once at the end."""
    k = position.shape[1]
    if k <= MAX_CHOICES:
        return expert_combine(gX, position.contiguous())
    rows, total = gX.float(), None
    for j in range(0, k, MAX_CHOICES):
        total = expert_combine(rows, position[:, j:j + MAX_CHOICES].contiguous(), base=total, out=total)
    return total.to(gX.dtype)


class Int8ExpertsFunction(torch.autograd.Function):
    """The experts' products in int8, with the memory-efficient input gradient: tokens (T x K) to rows (R x N).

    position (T x k): the rows of each token, needed for the gradient where `rows` is given. Each row's gradient is
    rounded to x's dtype, then a token's rows are added in fp32 and rounded again."""

    @staticmethod
    def forward(ctx, x, CB, SCB, seg_offsets, seg_expert, rows, position, threshold):
        X = x.contiguous()
        out = expert_forward(X, CB, SCB, seg_offsets, seg_expert, rows, threshold)
        ctx.save_for_backward(CB, SCB, seg_offsets, seg_expert, rows, position)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        CB, SCB, seg_offsets, seg_expert, rows, position = ctx.saved_tensors
        if not ctx.needs_input_grad[0]:
            return (None,) * 8
        if rows is not None and position is None:
            raise ValueError("the gradient of gathered tokens needs position, the rows of each token")
        gX = expert_backward(g.contiguous(), CB, SCB, seg_offsets, seg_expert)
        if rows is not None:
            gX = _sum_of_rows(gX, position)
        return gX, None, None, None, None, None, None, None


class ExpertCombineFunction(torch.autograd.Function):
    """Weighted sum of each token's rows plus base: gradients for the rows, the gate and base.

    Positions may be any: a row that several name gets the sum of their terms, a row that none names (also one whose
    position was taken out after the sort) 0. n_rows (the sort's last offset) is not needed for that; it may be None."""

    @staticmethod
    def forward(ctx, Y, position, gate, base, n_rows):
        Yc = Y.contiguous()
        gate_c = None if gate is None else gate.contiguous()
        out = expert_combine(Yc, position, gate_c, None if base is None else base.contiguous())
        ctx.rows = Y.shape[0]
        ctx.save_for_backward(Yc if gate is not None and ctx.needs_input_grad[2] else None, position, gate_c)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        Y, position, gate = ctx.saved_tensors
        need = ctx.needs_input_grad
        gY = gg = None
        if need[0] or need[2]:
            g2 = g.contiguous()
            gY, gg = expert_combine_backward(g2, position, gate, Y, rows=ctx.rows, with_grad_Y=need[0],
                                             with_grad_gate=need[2], any_positions=need[0])
        return gY, None, gg, g if need[3] else None, None


class Int8Experts(torch.nn.Module):
    """Projections of `experts` experts with frozen int8 weights (quantized once): weight is (experts, N, K)."""

    def __init__(self, weight: torch.Tensor, threshold: float = 6.0):
        super().__init__()
        from . import quantize_weight
        if weight.dim() != 3:
            raise ValueError("weight must be (experts, N, K)")
        E, N, K = weight.shape
        CB, SCB = quantize_weight(weight.detach().reshape(E * N, K).contiguous())
        self.register_buffer("CB", CB.view(E, N, K))
        self.register_buffer("SCB", SCB.view(E, N))
        self.threshold = float(threshold)

    def forward(self, x, seg_offsets, seg_expert=None, rows=None, position=None):
        """x: (T, K) -> (R, N), as expert_forward; position as Int8ExpertsFunction."""
        return Int8ExpertsFunction.apply(x, self.CB, self.SCB, seg_offsets, seg_expert, rows, position, self.threshold)
