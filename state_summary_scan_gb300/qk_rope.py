"""Norm of each head of queries and keys with the position rotation in the same pass.

The calls allocate outputs and issue rm_cp_qkr_forward / rm_cp_qkr_backward; `qk_norm_rope_train`
is the differentiable form.  `make_rope_table` computes the rotation's table once, in fp64.
"""
from __future__ import annotations

import collections
import ctypes
import math
import threading
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _capi as C

_NORMS = {"none": 0, "rms": 1, "l2": 2}
_DTYPES = {torch.float32: C.RM_F32, torch.bfloat16: C.RM_BF16}


def make_rope_table(max_positions: int, rotary_dim: int, base: float = 10000.0, scaling: str = "none",
                    factor: float = 1.0, trained_positions: Optional[int] = None, beta_fast: float = 32.0,
                    beta_slow: float = 1.0, device="cuda") -> torch.Tensor:
    """cos and sin of every position: [max_positions, 2, rotary_dim / 2] fp32.

    Pair i turns by base^(-2i / rotary_dim) a position.  scaling, for contexts `factor` times
    the trained one: "linear" divides every frequency by factor; "ntk" raises the base so that the
    slowest pair's frequency is divided by factor and the fastest is kept; "yarn" keeps pairs
    that turn at least beta_fast times over trained_positions, divides those that turn at most
    beta_slow times, blends between them, and scales cos and sin by 0.1 ln(factor) + 1.  The blend
    is linear in the turns of a pair; tables that blend over the pair's index differ between the two."""
    if rotary_dim <= 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be positive and even")
    if max_positions <= 0:
        raise ValueError("max_positions must be positive")
    if scaling not in ("none", "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if not factor >= 1.0:
        raise ValueError("factor must be at least 1")
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    mult = 1.0
    if scaling == "ntk" and rotary_dim > 2:
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    inv = float(base) ** (-2.0 * i / rotary_dim)
    if scaling == "linear":
        inv = inv / factor
    elif scaling == "yarn":
        if not trained_positions:
            raise ValueError("yarn scaling needs trained_positions")
        if not beta_fast > beta_slow:
            raise ValueError("beta_fast must be above beta_slow")
        turns = trained_positions * inv / (2 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0, 1)
        inv = inv * keep + inv / factor * (1 - keep)
        mult = 0.1 * math.log(factor) + 1.0
    angle = torch.arange(max_positions, dtype=torch.float64)[:, None] * inv
    return (torch.stack([angle.cos(), angle.sin()], 1) * mult).to(torch.float32).to(device).contiguous()


_CACHE: "collections.OrderedDict" = collections.OrderedDict()  # checked problems by signature
_CACHE_MAX = 256
_CACHE_LOCK = threading.Lock()


def _problem(q, k, table, positions, q_weight, k_weight, norm, eps, interleaved):
    """(problem, its address) of a call, checked once for each combination of shapes, strides,
    types and options."""
    sig = C.signature
    key = (sig(q), sig(k), sig(table), sig(positions), sig(q_weight), sig(k_weight), norm, eps, interleaved)
    hit = _CACHE.get(key)
    if hit is None:
        p = _checked_problem(q, k, table, positions, q_weight, k_weight, norm, eps, interleaved)
        hit = (p, ctypes.addressof(p))
        with _CACHE_LOCK:
            _CACHE[key] = hit
            while len(_CACHE) > _CACHE_MAX:
                _CACHE.popitem(last=False)
    return hit


def _checked_problem(q, k, table, positions, q_weight, k_weight, norm, eps, interleaved) -> C.QkrProblem:
    if q.dim() != 4 or k.dim() != 4 or q.shape[:2] != k.shape[:2] or q.shape[3] != k.shape[3]:
        raise ValueError("q and k must be [B,T,Hq,D] and [B,T,Hk,D]")
    if 0 in q.shape[2:] or 0 in k.shape[2:]:
        raise ValueError("q and k must have heads and elements")
    if q.dtype != k.dtype or q.dtype not in _DTYPES:
        raise ValueError("q and k must both be fp32 or both bf16")
    if not q.is_cuda or q.device != k.device:
        raise ValueError("q and k must be on one CUDA device")
    B, T, Hq, D = q.shape
    if q.stride(3) != 1 or k.stride(3) != 1:
        raise ValueError("the elements of a head of q and k must be adjacent")
    R = 0
    if table is not None:
        if table.dim() != 3 or table.shape[1] != 2 or table.dtype != torch.float32 or not table.is_contiguous():
            raise ValueError("the table must be [max_positions, 2, rotary_dim / 2] fp32, contiguous")
        if table.device != q.device:
            raise ValueError("the table must be on the device of q")
        R = 2 * table.shape[2]
    pos_rows = pos64 = 0
    if positions is not None:
        if positions.device != q.device or positions.dtype not in (torch.int32, torch.int64):
            raise ValueError("positions must be int32 or int64 on the device of q")
        if not positions.is_contiguous() or tuple(positions.shape) not in ((T,), (1, T), (B, T)):
            raise ValueError("positions must be [T] or [B,T], contiguous")
        pos_rows = B if tuple(positions.shape) == (B, T) else 1
        pos64 = int(positions.dtype == torch.int64)
    for w in (q_weight, k_weight):
        if w is not None and (w.dtype != torch.float32 or tuple(w.shape) != (D,) or not w.is_contiguous()
                              or w.device != q.device):
            raise ValueError("weights must be [D] fp32, contiguous, on the device of q")
    if norm not in _NORMS:
        raise ValueError(f"norm must be one of {sorted(_NORMS)}")

    def strides(x):  # a dimension of one element takes no step
        return tuple(0 if n == 1 else s for n, s in zip(x.shape[:3], x.stride()[:3]))

    return C.QkrProblem(B, T, Hq, k.shape[2], D, R, _NORMS[norm], int(bool(interleaved)), eps, _DTYPES[q.dtype],
                        table.shape[0] if table is not None else 0, pos_rows, pos64, strides(q), strides(k))


def qk_norm_rope(q, k, table=None, positions=None, q_weight=None, k_weight=None, norm: str = "rms", eps: float = 1e-6,
                 interleaved: bool = False, out=None, stream=None):
    """(q', k'): the norm of each head of q [B,T,Hq,D] and k [B,T,Hk,D] (norm "rms", "l2" or
    "none", times the weights [D] where given), then the rotation of the first rotary_dim
    elements by the table's rows at `positions` ([T] or [B,T]; None: 0 .. T-1).  table None: no
    rotation.  Pairs are (i, i + rotary_dim / 2), or (2i, 2i + 1) with interleaved.  q and k may
    be slices of a fused projection (adjacent elements, 16-byte strides); the outputs are
    contiguous and alias no input.  A position outside the table makes its token's rotated
    elements NaN."""
    _, p = _problem(q, k, table, positions, q_weight, k_weight, norm, eps, interleaved)
    if out is None:
        out = (_new(q), _new(k)) if stream is None else C.on_stream(lambda: (_new(q), _new(k)), stream, q.get_device())
    else:
        _like(out, (q, k), "out")
        C.written(out)
    if q.numel():
        C.rm_cp_qkr_forward(p, q, k, q_weight, k_weight, table, positions, out[0], out[1],
                            C._raw_stream(stream, q.get_device()))
    return out


def _new(x):
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _like(got, want, name):
    for x, y in zip(got, want):
        if x.shape != y.shape or x.dtype != y.dtype or x.device != y.device or not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous and have the shapes, type and device of q and k")


def qk_norm_rope_backward(q, k, dq_out, dk_out, table=None, positions=None, q_weight=None, k_weight=None,
                          norm: str = "rms", eps: float = 1e-6, interleaved: bool = False, stream=None):
    """(dq, dk, dq_weight, dk_weight) of sum(dq_out * q') + sum(dk_out * k'), with the arguments
    of the forward; a weight's gradient is [D] fp32, None without the weight."""
    problem, p = _problem(q, k, table, positions, q_weight, k_weight, norm, eps, interleaved)
    _like((dq_out, dk_out), (q, k), "dq_out and dk_out")
    size = C.rm_cp_qkr_workspace_size(problem) if q.numel() and (q_weight is not None or k_weight is not None) else 0

    def buffers():
        weight = torch.empty_like if q.numel() else torch.zeros_like  # no rows: their sum is 0
        return (_new(q), _new(k), None if q_weight is None else weight(q_weight), None if k_weight is None else weight(k_weight),
                torch.empty(size, dtype=torch.uint8, device=q.device) if size else None)

    dq, dk, dwq, dwk, ws = C.on_stream(buffers, stream, q.get_device())
    if not q.numel():
        return dq, dk, dwq, dwk
    C.rm_cp_qkr_backward(p, q, k, q_weight, k_weight, table, positions, dq_out, dk_out, dq, dk, dwq, dwk, ws,
                         C._raw_stream(stream, q.get_device()))
    return dq, dk, dwq, dwk


class QkNormRope(torch.autograd.Function):
    """Autograd adapter: the backward recomputes the norm from the saved q and k."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, table, positions, norm, eps, interleaved):
        ctx.save_for_backward(q, k, q_weight, k_weight, table, positions)
        ctx.how = dict(norm=norm, eps=eps, interleaved=interleaved)
        return qk_norm_rope(q, k, table, positions, q_weight, k_weight, **ctx.how)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, table, positions = ctx.saved_tensors
        dq, dk, dwq, dwk = qk_norm_rope_backward(q, k, dq_out.contiguous(), dk_out.contiguous(), table, positions,
                                                 q_weight, k_weight, **ctx.how)
        return dq, dk, dwq, dwk, None, None, None, None, None


def qk_norm_rope_train(q, k, table=None, positions=None, q_weight=None, k_weight=None, norm: str = "rms",
                       eps: float = 1e-6, interleaved: bool = False):
    """Differentiable qk_norm_rope (gradients of q, k and the weights)."""
    return QkNormRope.apply(q, k, q_weight, k_weight, table, positions, norm, eps, interleaved)
