"""Global norm of many gradient tensors, and clipping (rm_cp_clip_grad_norm)."""
from __future__ import annotations

import array
import dataclasses
import operator
from typing import Optional, Sequence

import torch

from . import _capi as C

_DTYPES = {torch.float32: C.RM_F32, torch.bfloat16: C.RM_BF16}


@dataclasses.dataclass
class ClipPlan:
    """Workspace of clip_grad_norm for up to max_tensors tensors; calls on one plan follow one
    another."""
    max_tensors: int
    device: torch.device
    ws: torch.Tensor


def make_clip_plan(max_tensors: int, device="cuda") -> ClipPlan:
    if max_tensors <= 0:
        raise ValueError("max_tensors must be positive")
    ws = torch.empty(C.rm_cp_clip_workspace_size(max_tensors), dtype=torch.uint8, device=device)
    return ClipPlan(max_tensors, ws.device, ws)


_DTYPE = operator.attrgetter("dtype")
_Tensor = torch.Tensor


def _describe(tensors, device, name):
    """Addresses and type codes of contiguous fp32 or bf16 tensors on one device."""
    try:
        types = array.array("i", map(_DTYPES.__getitem__, map(_DTYPE, tensors)))
    except KeyError as e:
        raise ValueError(f"{name} must be fp32 or bf16, not {e.args[0]}") from None
    if set(map(_Tensor.get_device, tensors)) != {device.index}:
        raise ValueError(f"{name} must be on the plan's device")
    if not all(map(_Tensor.is_contiguous, tensors)):
        raise ValueError(f"{name} must be contiguous")
    return array.array("Q", map(_Tensor.data_ptr, tensors)), types


def clip_grad_norm(plan: ClipPlan, grads: Sequence[torch.Tensor], max_norm: Optional[float] = None, out=None,
                   eps: float = 1e-6, stream=None) -> torch.Tensor:
    """The 2-norm over every element of grads (a fp32 scalar on the device, no host read).  With
    max_norm each gradient is multiplied by min(1, max_norm / (norm + eps)), in place or, with
    out, into the tensors of out (same sizes, fp32 or bf16 each; gradients can be cast on the
    way); a tensor that is written may not overlap any other.  grads: contiguous fp32 and bf16 tensors of any sizes and alignments, mixed."""
    grads = grads if isinstance(grads, (list, tuple)) else list(grads)
    if not grads:
        raise ValueError("no gradients")
    if len(grads) > plan.max_tensors:
        raise ValueError(f"{len(grads)} tensors exceed the plan's {plan.max_tensors}")
    ptr, types = _describe(grads, plan.device, "gradients")
    sizes = array.array("q", map(_Tensor.numel, grads))
    out_ptr, out_types = ptr, types
    if out is not None:
        if max_norm is None:
            raise ValueError("out needs max_norm")
        if array.array("q", map(_Tensor.numel, out)) != sizes:
            raise ValueError("out must have the sizes of the gradients")
        out_ptr, out_types = _describe(out, plan.device, "out")
    if stream is None:
        norm = torch.empty((), dtype=torch.float32, device=plan.device)
    else:
        norm = C.on_stream(lambda: torch.empty((), dtype=torch.float32, device=plan.device), stream, plan.device.index)

    def at(a):
        return a.buffer_info()[0]

    C.rm_cp_clip_grad_norm(len(grads), at(ptr), at(sizes), at(types), None if max_norm is None else at(out_ptr),
                           None if max_norm is None else at(out_types), 0.0 if max_norm is None else max_norm, eps, norm,
                           plan.ws, C._raw_stream(stream, plan.device.index))
    if max_norm is not None:
        C.written(grads if out is None else out)
    return norm
