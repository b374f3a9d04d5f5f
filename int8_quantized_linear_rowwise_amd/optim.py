"""AdamW over many tensors in one launch, with states in 32 or in 8 bits:
binding of int8_adamw_* (include/int8lin.h) and an optimizer.

8-bit states are float8_e4m3fn tensors with one power-of-two fp32 scale for
each block of 256 values: m = code * scale, and the second tensor holds the
root, sqrt(v) = code * scale.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence, Tuple

import torch

from ._lib import AdamWTensor, check, lib
from ._tensors import DTYPE_CODE, _on_gpu, _ptr, _raw_stream
from .grad_norm import GradNormPlan

BLOCK = 256   # values that share a scale


def _capturing(dev: int) -> bool:
    """Whether the current stream of GPU number `dev` is being captured into a graph."""
    if dev < 0:
        return False
    with _on_gpu(dev):
        return torch.cuda.is_current_stream_capturing()


def _check_numbers(lr, betas, eps, weight_decay, state_bits=32, **other) -> None:
    for name, x in (("lr", lr), ("eps", eps), ("weight_decay", weight_decay)):
        if not (0.0 <= x < math.inf):
            raise ValueError(f"{name} must be a finite number of 0 or more, got {x}")
    if len(betas) != 2 or not all(0.0 <= b < 1.0 for b in betas):
        raise ValueError(f"betas must be two numbers in [0, 1), got {betas}")
    if state_bits not in (8, 32):
        raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")


def adamw_state(p: torch.Tensor, bits: int = 32, master: bool = False) -> dict:
    """The state of one parameter before the first step: m, v, for 8 bits their scales, and the fp32 master copy
    if asked for."""
    if bits not in (8, 32):
        raise ValueError("state bits must be 8 or 32")
    n, dev = p.numel(), p.device
    if bits == 32:
        s = {"m": torch.zeros(p.shape, dtype=torch.float32, device=dev),
             "v": torch.zeros(p.shape, dtype=torch.float32, device=dev)}
    else:
        blocks = -(-n // BLOCK)
        s = {"m": torch.zeros(p.shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn),
             "v": torch.zeros(p.shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn),
             "m_scale": torch.zeros(blocks, dtype=torch.float32, device=dev),
             "v_scale": torch.zeros(blocks, dtype=torch.float32, device=dev)}
    if master:
        s["master"] = p.detach().to(torch.float32, copy=True)
    return s


class AdamWPlan:
    """The tensors of an AdamW step, checked and laid out on the device once; `step` is one launch.

    params, grads: tensors of one dtype each pair (fp32, fp16 or bf16); m, v:
    their states, all fp32 or all float8_e4m3fn (then with m_scale and v_scale);
    master: fp32 copies or None. The plan reads and writes these very tensors
    at every step (grads have to be filled in place) and keeps them alive."""

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], m: Sequence[torch.Tensor],
                 v: Sequence[torch.Tensor], m_scale: Optional[Sequence[torch.Tensor]] = None,
                 v_scale: Optional[Sequence[torch.Tensor]] = None,
                 master: Optional[Sequence[torch.Tensor]] = None):
        n = len(params)
        lists = dict(grads=grads, m=m, v=v, m_scale=m_scale, v_scale=v_scale, master=master)
        for name, x in lists.items():
            if x is not None and len(x) != n:
                raise ValueError(f"{name} must have one tensor for each of the {n} parameters")
        if n == 0:
            raise ValueError("no parameters")
        self.device, self.gpu = params[0].device, params[0].get_device()
        self._keep = [list(params)] + [list(x) for x in lists.values() if x is not None]
        self.table, self.count, self.chunks = None, n, 0
        arr = (AdamWTensor * n)()
        none = [None] * n
        names = ("params", "grads", "m", "v", "m_scale", "v_scale", "master")
        for i, row in enumerate(zip(params, grads, m, v, m_scale or none, v_scale or none, master or none)):
            p, g, mi, vi, ms, vs, w = row
            size, dtype = p.numel(), p.dtype
            low = mi.dtype == torch.float8_e4m3fn
            state = torch.float8_e4m3fn if low else torch.float32
            if dtype not in DTYPE_CODE:
                raise TypeError(f"unsupported dtype {dtype}; expected float32, float16 or bfloat16")
            if g.dtype != dtype or g.numel() != size:
                raise ValueError(f"grads[{i}] must have its parameter's size and dtype")
            if mi.dtype != state or vi.dtype != state or mi.numel() != size or vi.numel() != size:
                raise ValueError(f"m[{i}] and v[{i}] must both be float32 or both float8_e4m3fn, of the "
                                 "parameter's size")
            if low:
                for name, x in (("m_scale", ms), ("v_scale", vs)):
                    if x is None or x.dtype != torch.float32 or x.numel() != -(-size // BLOCK):
                        raise ValueError(f"{name}[{i}] must be float32 with one value for each {BLOCK}")
            else:
                row = (p, g, mi, vi, None, None, w)
            if w is not None and (w.dtype != torch.float32 or w.numel() != size):
                raise ValueError(f"master[{i}] must be float32 of the parameter's size")
            if self.gpu < 0:
                raise ValueError("parameters must be on a GPU")
            arr[i] = AdamWTensor(*[_ptr(t, k, self.gpu) or None for t, k in zip(row, names)], size,
                                 DTYPE_CODE[dtype], 8 if low else 32)
        if _capturing(self.gpu):
            raise RuntimeError("AdamW: the plan of a captured step has to be laid out before the capture (for the "
                               "optimizer: one ordinary step with the same gradients)")
        need = lib.int8_adamw_table_bytes(arr, n)
        host = torch.zeros(max(need, 1), dtype=torch.uint8)
        chunks = ctypes.c_int64(0)
        check(lib.int8_adamw_table_fill(arr, n, host.data_ptr(), need, ctypes.byref(chunks)), "int8_adamw_table_fill")
        self.chunks = chunks.value
        self.table = host.to(self.device)
        self._stream = _raw_stream(self.gpu)

    def _scalar(self, x: Optional[torch.Tensor], name: str) -> int:
        """Device pointer of one of the step's two scalars, 0 for None."""
        if x is None:
            return 0
        if x.dtype != torch.float32 or x.numel() != 1 or x.get_device() != self.gpu:
            raise ValueError(f"{name} must be one float32 value on {self.device}")
        return x.data_ptr()

    def step(self, step: int, lr: float, betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
             weight_decay: float = 0.01, grad_scale: Optional[torch.Tensor] = None,
             found_inf: Optional[torch.Tensor] = None) -> None:
        """Step number `step` (from 1). grad_scale: fp32 GPU scalar that multiplies the gradients; found_inf: fp32 GPU
        scalar, anything but 0 leaves all tensors as they are (the caller's step count goes on). A captured step keeps
        its numbers; only the two scalars are read at each replay: the caller keeps them, and the plan, as long
        as the graph."""
        scale, inf = self._scalar(grad_scale, "grad_scale"), self._scalar(found_inf, "found_inf")
        stream = _raw_stream(self.gpu)
        if stream != self._stream:     # the table's memory is not given away before this stream is done with it
            self.table.record_stream(torch.cuda.current_stream(self.device))
        with _on_gpu(self.gpu):
            check(lib.int8_adamw_step(self.table.data_ptr(), self.count, self.chunks, lr, betas[0], betas[1], eps,
                                      weight_decay, step, scale, inf, stream),
                  "int8_adamw_step")


class AdamW(torch.optim.Optimizer):
    """AdamW with every parameter of a group updated in one launch.

    state_bits: 32 or 8; master: keep fp32 copies of fp16 / bf16 parameters.
    The plan of a group is laid out again whenever a gradient or parameter has
    moved (gradients kept in place with zero_grad(set_to_none=False) never do): a
    step of 448 tensors takes the host 0.5 ms, 2.3 ms where it is laid out again.
    Parameters and gradients have to be contiguous. A captured step keeps its
    step number and learning rate; what it uses is held as long as the optimizer.
    One ordinary step with the same gradients comes before a capture: it makes the
    states and lays out the plan."""

    def __init__(self, params, lr: float = 1e-3, betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.01, state_bits: int = 32, master: bool = False):
        defaults = dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, state_bits=state_bits, master=master)
        _check_numbers(**defaults)
        super().__init__(params, defaults)
        self._plans: dict = {}
        self._captured: list = []

    def add_param_group(self, param_group):
        _check_numbers(**{**self.defaults, **param_group})
        super().add_param_group(param_group)

    def __setstate__(self, state):
        """Plans name the addresses of the states before: a copy, an unpickled optimizer and load_state_dict, which
        comes through here too, start without. What this optimizer's own captured steps use stays held."""
        super().__setstate__(state)
        self._plans = {}
        self.__dict__.setdefault("_captured", [])

    @torch.no_grad()
    def step(self, closure=None, grad_scale: Optional[torch.Tensor] = None, found_inf: Optional[torch.Tensor] = None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        # everything is checked and laid out before the first launch: a refused step changes nothing
        due, plans = [], {}
        for gi, group in enumerate(self.param_groups):
            _check_numbers(**group)
            buckets: dict = {}
            for p in group["params"]:
                if p.grad is None:
                    continue
                s = self.state.get(p)
                if not s:
                    if _capturing(p.get_device()):   # the zeros would be written again at every replay
                        raise RuntimeError("AdamW: states have to be made before the capture: take one ordinary step "
                                           "with the same gradients first")
                    s = adamw_state(p, group["state_bits"], group["master"] and p.dtype != torch.float32)
                    s["step"] = 0
                buckets.setdefault((p.device, s["step"] + 1, "master" in s), []).append((p, p.grad, s))
            live = plans[gi] = {}
            for (device, step, has_master), rows in buckets.items():
                where = tuple(x.data_ptr() for p, g, s in rows
                              for x in (p, g, s["m"], s["v"], s.get("m_scale"), s.get("v_scale"), s.get("master"))
                              if x is not None)
                where += tuple((p.numel(), p.dtype, g.dtype, p.is_contiguous(), g.is_contiguous()) for p, g, s in rows)
                key = (device, has_master, tuple(id(r[0]) for r in rows))
                held = self._plans.get(gi, {}).get(key)
                if held is None or held[0] != where:
                    low = group["state_bits"] == 8
                    held = (where, AdamWPlan(
                        [r[0].detach() for r in rows], [r[1] for r in rows], [r[2]["m"] for r in rows],
                        [r[2]["v"] for r in rows], [r[2]["m_scale"] for r in rows] if low else None,
                        [r[2]["v_scale"] for r in rows] if low else None,
                        [r[2]["master"] for r in rows] if has_master else None))
                    # every step compares the addresses: old gradients need not be held (their memory is the next
                    # backward pass's where zero_grad drops them)
                    held[1]._keep = None
                held[1]._scalar(grad_scale, "grad_scale"), held[1]._scalar(found_inf, "found_inf")
                live[key] = held
                due.append((held[1], step, group, rows))
        for plan, step, group, rows in due:
            if _capturing(plan.gpu):   # a graph's replays use the table, these very tensors and the two scalars
                self._captured.append((plan, [(p.detach(), g, dict(s)) for p, g, s in rows], grad_scale, found_inf))
            plan.step(step, group["lr"], group["betas"], group["eps"], group["weight_decay"], grad_scale, found_inf)
            for p, _, s in rows:
                s["step"] = step
                if step == 1:
                    self.state[p] = s
        self._plans = plans
        return loss

    def grad_norm(self, max_norm: Optional[float] = None, norm_type: float = 2.0,
                  grad_scale: Optional[torch.Tensor] = None):
        """(norm, factor, found_inf) over the gradients of all groups, as GradNormPlan.norm: `step` takes the factor as
        its grad_scale, which clips without a pass of its own, and found_inf. There has to be a gradient, and all of
        them on one GPU. The list is laid out at every call (0.24 ms of host time for 448 tensors; a GradNormPlan over
        gradients that stay in place is laid out once)."""
        grads = [p.grad for group in self.param_groups for p in group["params"] if p.grad is not None]
        plan = GradNormPlan(grads)
        if _capturing(plan.gpu):   # a graph's replays read these very gradients and the scale
            self._captured.append((plan, grad_scale))
        return plan.norm(max_norm, norm_type, grad_scale)

    def load_state_dict(self, state_dict):
        """States keep their own types (the base class would turn them into the parameter's)."""
        super().load_state_dict(state_dict)
        saved = state_dict["state"]
        ids = [i for g in state_dict["param_groups"] for i in g["params"]]
        params = [p for g in self.param_groups for p in g["params"]]
        for i, p in zip(ids, params):
            for k, x in saved.get(i, {}).items():
                if isinstance(x, torch.Tensor):
                    self.state[p][k] = x.detach().to(p.device, copy=True)
        self._plans = {}
