"""Root-mean-square norm of rows around a mixer: with the residual's addition before it, a gate (the norm of a
mixer's outputs), and an output in 8 bits with scales for the projection behind it.

The calls allocate outputs and issue rm_cp_rms_forward / rm_cp_rms_quant / rm_cp_rms_backward;
`rms_norm_train` is the differentiable form.
"""
from __future__ import annotations

import collections
import ctypes
import math
import threading

import torch
from torch.autograd.function import once_differentiable

from . import _capi as C

_DTYPES = {torch.float32: C.RM_F32, torch.bfloat16: C.RM_BF16}
_CACHE: "collections.OrderedDict" = collections.OrderedDict()  # checked problems by signature
_CACHE_MAX = 256
_CACHE_LOCK = threading.Lock()


def _steps(t, first, last):
    """The stride of dimensions [first, last) of t taken as one, or None where they have no single one."""
    step = want = None  # (a broadcast dimension's step is 0: none yet is not the same)
    for n, s in reversed(list(zip(t.shape[first:last], t.stride()[first:last]))):
        if n == 1:
            continue  # (takes no step)
        if want is not None and s != want:
            return None
        step, want = s if step is None else step, s * n
    return step or 0


def _rows(tensors):
    """(N, H, strides of each tensor): the rows of tensors [..., n] of one shape as N tokens of H rows."""
    shape = tensors[0].shape[:-1]
    if 0 in shape:
        return 0, 1, [(0, 0)] * len(tensors)
    for at in range(len(shape), -1, -1):
        strides = [(_steps(t, 0, at), _steps(t, at, len(shape))) for t in tensors]
        if all(None not in s for s in strides):
            return math.prod(shape[:at]), math.prod(shape[at:]), strides
    raise ValueError("the rows of every tensor must be evenly spaced in at most two dimensions")


def _problem(x, residual, weight, gate, gate_first, group, eps, dy=None, dh=None):
    """(problem, its address, shape of its scales), checked once for each combination of shapes, strides, types and options.
    The caller holds the problem until its C call has returned: another thread's calls may push it out of the cache."""
    sig = C.signature
    key = (sig(x), sig(residual), sig(weight), sig(gate), gate_first, group, eps, sig(dy), sig(dh))
    hit = _CACHE.get(key)
    if hit is None:
        p = _checked_problem(x, residual, weight, gate, gate_first, group, eps, dy, dh)
        hit = (p, ctypes.addressof(p), torch.Size((*x.shape[:-1], p.n // group if group else 1)))
        with _CACHE_LOCK:
            _CACHE[key] = hit
            while len(_CACHE) > _CACHE_MAX:
                _CACHE.popitem(last=False)
    return hit


def _checked_problem(x, residual, weight, gate, gate_first, group, eps, dy, dh) -> C.RmsProblem:
    """x: the rows (in a backward: h, and residual None)."""
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError("x must have rows of elements")
    if x.dtype not in _DTYPES or (residual is not None and residual.dtype not in _DTYPES):
        raise ValueError("x and the residual must be fp32 or bf16")
    if not x.is_cuda:
        raise ValueError("x must be on a CUDA device")
    if residual is not None and gate is not None:
        raise ValueError("a residual and a gate exclude one another")
    if gate_first and gate is None:
        raise ValueError("gate_first needs a gate")
    others = [t for t in (residual, gate, dy, dh) if t is not None]
    if any(t.shape != x.shape for t in others):
        raise ValueError("the residual, the gate and the gradients must have the shape of x")
    if any(t.device != x.device for t in others + ([weight] if weight is not None else [])):
        raise ValueError("every tensor must be on the device of x")
    dtype, res_dtype = x.dtype, x.dtype
    if residual is not None:
        res_dtype = residual.dtype
    if dy is not None:
        if dy.dtype not in _DTYPES or not dy.is_contiguous():
            raise ValueError("dy must be fp32 or bf16, contiguous")
        dtype = dy.dtype
        if dh is not None and (dh.dtype != x.dtype or not dh.is_contiguous()):
            raise ValueError("dh must have the type of h, contiguous")
    if dtype == torch.float32 and res_dtype != torch.float32:
        raise ValueError("fp32 rows need an fp32 residual")
    if gate is not None and (gate.dtype != dtype or res_dtype != dtype):
        raise ValueError("the gate must have the type of x")
    n = x.shape[-1]
    if weight is not None and (weight.dtype != torch.float32 or tuple(weight.shape) != (n,) or not weight.is_contiguous()):
        raise ValueError("the weight must be [n] fp32, contiguous")
    for t, name in ((x, "x"), (residual, "the residual"), (gate, "the gate")):
        if t is not None and n > 1 and t.stride(-1) != 1:
            raise ValueError(f"the elements of a row of {name} must be adjacent")
    N, H, strides = _rows([t for t in (x, residual, gate) if t is not None])
    zero = (0, 0)
    xs = strides[0]
    rs = strides[1] if residual is not None else xs  # (in a backward h takes the residual's place)
    zs = strides[-1] if gate is not None else zero
    if N > (1 << 31) - 1 or H > (1 << 31) - 1:
        raise ValueError("too many rows")
    return C.RmsProblem(N, max(H, 1), n, eps, _DTYPES[dtype], _DTYPES[res_dtype], 0 if gate is None else 2 if gate_first else 1, group,
                        zero if dy is not None else xs, rs, zs)


def _new(x):
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _given(t, like, dtype, name):
    if t.shape != like.shape or t.dtype != dtype or t.device != like.device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, {dtype}, and have the shape and device of x")


def _check_given(x, residual, h, out, dtype):
    if h is not None:
        if residual is None:
            raise ValueError("h needs a residual")
        _given(h, residual, residual.dtype, "h")
    if out is not None:
        _given(out, x, dtype, "out")


def rms_norm(x, weight=None, residual=None, gate=None, gate_first: bool = False, eps: float = 1e-6, out=None, h=None,
             stream=None):
    """(y, h): y = u (mean(u^2) + eps)^(-1/2) weight over the last dimension of x [..., n].

    residual [..., n]: u = h = x + residual, rounded to the residual's type; it goes into a new tensor, or into h,
    which may be the residual itself (the residual stream updated in place).  Without one h is x.
    gate [..., n] (the norm of a mixer's outputs): y is times gate sigmoid(gate), or, with gate_first, u = x gate
    sigmoid(gate).  x and y are fp32 or bf16, the residual of x's type or fp32, the gate of x's type, the weight
    [n] fp32.  x, residual and gate may be slices of a fused projection (adjacent elements, 16-byte bases and strides, rows
    evenly spaced in at most two dimensions); y and h are contiguous, and y may go into a contiguous x (out=x).
    n is a multiple of 8 up to 32768."""
    p, at, _ = _problem(x, residual, weight, gate, gate_first, 0, eps)
    device = x.get_device()
    if out is not None or h is not None:
        _check_given(x, residual, h, out, x.dtype)
        C.written([t for t in (out, h) if t is not None])

    def buffers():
        return _new(x) if out is None else out, x if residual is None else _new(residual) if h is None else h

    y, total = buffers() if stream is None else C.on_stream(buffers, stream, device)
    if x.numel():
        C.rm_cp_rms_forward(at, x, residual, gate, weight, total if residual is not None else None, y, C._raw_stream(stream, device))
    return y, total


def rms_norm_quant(x, weight=None, residual=None, gate=None, gate_first: bool = False, group: int = 0, eps: float = 1e-6,
                   out=None, h=None, stream=None):
    """(y8, scales, h): rms_norm with y in 8 bits, y8 [..., n] e4m3 and scales [..., n / group] fp32 with y ~ y8 scale.

    A scale is max |y| / 448 of `group` adjacent elements (32, 64 or 128; 0: of the row), at least 2^-126; y is not
    rounded before it is divided by it.  out: (y8, scales) to write into.  A row with a NaN in u has NaN scales; a NaN in the weight,
    or in a gate behind the norm, makes its element of y8 NaN."""
    p, at, scale_shape = _problem(x, residual, weight, gate, gate_first, group, eps)
    device = x.get_device()
    if out is not None or h is not None:
        _check_given(x, residual, h, None if out is None else out[0], torch.float8_e4m3fn)
        if out is not None and (out[1].shape != scale_shape or out[1].dtype != torch.float32 or out[1].device != x.device or not out[1].is_contiguous()):
            raise ValueError(f"out[1] must be {list(scale_shape)} fp32, contiguous, on the device of x")
        C.written([t for t in (*(out or ()), h) if t is not None])

    def buffers():
        total = x if residual is None else _new(residual) if h is None else h
        if out is not None:
            return out[0], out[1], total
        return (torch.empty_like(x, dtype=torch.float8_e4m3fn, memory_format=torch.contiguous_format),
                torch.empty(scale_shape, dtype=torch.float32, device=x.device), total)

    y8, scales, total = buffers() if stream is None else C.on_stream(buffers, stream, device)
    if x.numel():
        C.rm_cp_rms_quant(at, x, residual, gate, weight, total if residual is not None else None, y8, scales, C._raw_stream(stream, device))
    return y8, scales, total


def rms_norm_backward(h, dy, weight=None, dh=None, gate=None, gate_first: bool = False, eps: float = 1e-6, stream=None):
    """(dx, dresidual, dgate, dweight) of sum(dy * y) + sum(dh * h), from the h that rms_norm gave (x where there was
    no residual).  dh: the gradient that comes down the residual stream, or None.  dx has the type of dy; dresidual
    is the same values in the type of h (dx itself where the types are equal); dgate (None without a gate) has the
    type of dy; dweight is [n] fp32, None without the weight.  dy and dh are contiguous."""
    p, at, _ = _problem(h, None, weight, gate, gate_first, 0, eps, dy, dh)
    device = h.get_device()
    size = C.rm_cp_rms_workspace_size(p) if weight is not None else 0

    def buffers():
        dx = _new(dy)
        return (dx, dx if h.dtype == dy.dtype else _new(h), None if gate is None else _new(dy),
                None if weight is None else torch.empty_like(weight),
                torch.empty(size, dtype=torch.uint8, device=h.device) if size else None)

    dx, dresidual, dgate, dweight, ws = buffers() if stream is None else C.on_stream(buffers, stream, device)
    if h.numel() or weight is not None:
        C.rm_cp_rms_backward(at, h, gate, weight, dy, dh, dx, dresidual, dgate, dweight, ws, C._raw_stream(stream, device))
    return dx, dresidual, dgate, dweight


def _dense(t):
    """t contiguous and from a 16-byte boundary on: autograd hands over contiguous views at any offset (of a concatenation's
    gradient)."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class RmsNorm(torch.autograd.Function):
    """Autograd adapter: the backward recomputes the norm from the saved h."""

    @staticmethod
    def forward(ctx, x, weight, residual, gate, gate_first, eps):
        ctx.set_materialize_grads(False)
        ctx.how = dict(gate_first=gate_first, eps=eps)
        y, h = rms_norm(x, weight, residual, gate, **ctx.how)
        ctx.save_for_backward(h, weight, gate)
        ctx.has_residual, ctx.dtype = residual is not None, x.dtype
        return (y, h) if residual is not None else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight, gate = ctx.saved_tensors
        if dy is None:  # y is not used
            return (None if dh is None else dh.to(ctx.dtype)), None, dh, None, None, None
        dx, dresidual, dgate, dweight = rms_norm_backward(h, _dense(dy), weight, None if dh is None else _dense(dh), gate, **ctx.how)
        return dx, dweight, dresidual if ctx.has_residual else None, dgate, None, None


def rms_norm_train(x, weight=None, residual=None, gate=None, gate_first: bool = False, eps: float = 1e-6):
    """Differentiable rms_norm: (y, h), with gradients of x, the weight, the residual and the gate."""
    got = RmsNorm.apply(x, weight, residual, gate, gate_first, eps)
    return got if residual is not None else (got, x)
