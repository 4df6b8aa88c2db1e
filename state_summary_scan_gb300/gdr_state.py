"""The gated delta rule with a carried state: ragged prefill and recurrent decoding on a pool of
states [num_slots, H, Dk, Dv] that the calls update in place (rm_gdr_state_forward).

`gated_delta_rule` trains the same recurrence over equal segments; these calls continue it one
prompt, or one token, at a time.
"""
from __future__ import annotations

import ctypes
import dataclasses
import math
from typing import Optional

import torch

from . import _capi as C

_DTYPES = {torch.float32: C.RM_F32, torch.bfloat16: C.RM_BF16}


@dataclasses.dataclass
class GdrStatePlan:
    """Sizes, bounds and workspace of a stream of calls on one pool.  Calls on one plan follow
    one another: they share its workspace."""
    c: C.GdrStateProblem
    max_seqs: int
    max_tokens: int
    max_len: int
    dtype: torch.dtype
    state_dtype: torch.dtype
    ws: torch.Tensor
    checked: dict = dataclasses.field(default_factory=dict)  # problems of calls by signature


def make_gdr_state_plan(max_seqs: int, max_tokens: int, H: int, Dk: int, Dv: int, num_slots: Optional[int] = None,
                        qk_heads: int = 0, max_len: Optional[int] = None, scale=None, dtype=torch.bfloat16,
                        state_dtype=torch.float32, device="cuda", recurrent: bool = False) -> GdrStatePlan:
    """Plan of calls with up to max_seqs sequences, max_tokens tokens in all and max_len tokens a
    sequence (default max_tokens).  qk_heads > 0: q and k have that many heads, each shared by
    H / qk_heads consecutive heads.  bf16 calls of 48 tokens a sequence or more (Dk 64 or 128) run in
    chunks on the tensor cores, which rounds some factors to bf16: outputs are off by up to one and a
    half times their own rounding, the state by some 1e-4 (2e-3 where a short prompt meets a state
    far larger than its values).  recurrent=True keeps every call a token
    recurrence at fp32's precision, whatever the lengths of its batch, and slower for prompts."""
    if dtype not in _DTYPES or state_dtype not in _DTYPES:
        raise ValueError("dtype and state_dtype must be fp32 or bf16")
    if scale is None:
        scale = 1.0 / math.sqrt(Dk)
    if max_len is None:
        max_len = max_tokens
    qk_heads = qk_heads or H
    c = C.GdrStateProblem(max_seqs, max_tokens, max_len, H, qk_heads, Dk, Dv, num_slots or max_seqs, scale,
                          _DTYPES[dtype], _DTYPES[state_dtype])
    c.q_stride = c.k_stride = (qk_heads * Dk, Dk)
    c.v_stride = (H * Dv, Dv)
    c.g_stride = c.beta_stride = H
    c.recurrent = int(recurrent)
    need = C.rm_gdr_state_workspace_size(c)
    if need == 0:
        raise C.RmCpError(C.load().rm_gdr_state_forward(c, *[None] * 12), C.load().rm_cp_last_error().decode())
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    return GdrStatePlan(c, max_seqs, max_tokens, max_len, dtype, state_dtype, ws)


def make_gdr_state(plan: GdrStatePlan) -> torch.Tensor:
    """A pool of zero states for the plan."""
    return torch.zeros(plan.c.num_slots, plan.c.H, plan.c.Dk, plan.c.Dv, dtype=plan.state_dtype, device=plan.ws.device)


def _strides(x, lead, name):
    """(token, head) strides of x [*lead, heads, D]; the tokens must be evenly spaced.  A dimension of one
    element takes no step, whatever its stride."""
    if x.stride(-1) != 1 and x.shape[-1] != 1:
        raise ValueError(f"the elements of a head of {name} must be adjacent")
    return _token_stride(x, lead, name), x.stride(-2) if x.shape[-2] > 1 else 0


def _token_stride(x, lead, name):
    if lead == 1:
        return x.stride(0) if x.shape[0] > 1 else 0
    S, n = x.shape[0], x.shape[1]
    if S > 1 and n > 1 and x.stride(0) != n * x.stride(1):
        raise ValueError(f"the tokens of {name} must be evenly spaced")
    return x.stride(1) if n > 1 else x.stride(0) if S > 1 else 0


def _checked_problem(plan, lead, S, N, max_len, q, k, v, g, beta, state, cu, slots, fresh):
    c, dev = plan.c, plan.ws.device
    head = q.shape[:lead]
    if (q.shape != (*head, c.qk_heads, c.Dk) or k.shape != q.shape or v.shape != (*head, c.H, c.Dv)
            or g.shape != (*head, c.H) or beta.shape != g.shape):
        raise ValueError(f"q and k must be [...,{c.qk_heads},{c.Dk}], v [...,{c.H},{c.Dv}], g and beta [...,{c.H}]")
    if q.dtype != plan.dtype or k.dtype != plan.dtype or v.dtype != plan.dtype:
        raise ValueError(f"q, k and v must be {plan.dtype}")
    if g.dtype != torch.float32 or beta.dtype != torch.float32:
        raise ValueError("g and beta must be fp32")
    if state.dtype != plan.state_dtype or state.shape != (c.num_slots, c.H, c.Dk, c.Dv) or not state.is_contiguous():
        raise ValueError(f"state must be [{c.num_slots},{c.H},{c.Dk},{c.Dv}] {plan.state_dtype}, contiguous")
    for x in (q, k, v, g, beta, state, cu, slots, fresh):
        if x is not None and x.device != dev:
            raise ValueError("every tensor must be on the plan's device")
    if S > plan.max_seqs or N > plan.max_tokens or max_len > plan.max_len:
        raise ValueError(f"{S} sequences, {N} tokens, {max_len} a sequence exceed the plan's "
                         f"{plan.max_seqs}, {plan.max_tokens}, {plan.max_len}")
    if slots is not None and (slots.dtype != torch.int32 or slots.shape != (S,) or not slots.is_contiguous()):
        raise ValueError("slots must be [sequences] int32, contiguous")
    if fresh is not None and (fresh.dtype not in (torch.uint8, torch.bool) or fresh.shape != (S,) or not fresh.is_contiguous()):
        raise ValueError("fresh must be [sequences] uint8 or bool, contiguous")
    if (g.stride(-1) != 1 or beta.stride(-1) != 1) and c.H > 1:
        raise ValueError("the heads of g and beta must be adjacent")
    p = C.GdrStateProblem.from_buffer_copy(c)
    p.num_seqs, p.num_tokens, p.max_len = S, N, max_len
    p.q_stride, p.k_stride, p.v_stride = _strides(q, lead, "q"), _strides(k, lead, "k"), _strides(v, lead, "v")
    p.g_stride, p.beta_stride = _token_stride(g, lead, "g"), _token_stride(beta, lead, "beta")
    return p


def _new(v):
    return torch.empty_like(v, memory_format=torch.contiguous_format)


def _call(plan, lead, S, N, max_len, q, k, v, g, beta, state, cu, slots, fresh, o, stream):
    sig = C.signature
    key = (lead, max_len, sig(q), sig(k), sig(v), sig(g), sig(beta), sig(state), sig(cu), sig(slots), sig(fresh))
    p = plan.checked.get(key)
    if p is None:
        p = _checked_problem(plan, lead, S, N, max_len, q, k, v, g, beta, state, cu, slots, fresh)
        if len(plan.checked) >= 256:
            plan.checked.clear()
        plan.checked[key] = p
    given = [state]
    if o is None:
        o = _new(v) if stream is None else C.on_stream(lambda: _new(v), stream, v.get_device())
    elif o.shape != v.shape or o.dtype != v.dtype or o.device != v.device or not o.is_contiguous():
        raise ValueError("o must be contiguous and have the shape, type and device of v")
    else:
        given.append(o)
    C.written(given)
    if S:
        C.rm_gdr_state_forward(ctypes.addressof(p), q, k, v, g, beta, cu, slots, fresh, state, o, plan.ws,
                               C._raw_stream(stream, q.get_device()))
    else:
        C.on_stream(o.zero_, stream, o.get_device())
    return o


def gdr_decode(plan: GdrStatePlan, q, k, v, g, beta, state, slots=None, fresh=None, o=None, stream=None) -> torch.Tensor:
    """o [S,n,H,Dv] of n tokens for each of S sequences, q, k [S,n,qk_heads,Dk], v [S,n,H,Dv], g,
    beta [S,n,H] fp32; the states of `state` at slots [S] int32 (None: 0 .. S-1) are updated in
    place.  A slot outside the pool marks a padding sequence (outputs 0).  fresh [S]: non-zero
    starts from a zero state.  q, k, v may be slices of a fused projection."""
    if q.dim() != 4:
        raise ValueError("q must be [sequences, tokens, heads, Dk]")
    S, n = q.shape[:2]
    return _call(plan, 2, S, S * n, n, q, k, v, g, beta, state, None, slots, fresh, o, stream)


def gdr_prefill(plan: GdrStatePlan, q, k, v, g, beta, state, cu_seqlens, slots=None, fresh=None, max_len=None, o=None,
                stream=None) -> torch.Tensor:
    """o [N,H,Dv] of S ragged prompts packed along N tokens; cu_seqlens [S + 1] int32 on the
    device.  max_len, a bound of the longest prompt (default the plan's), chooses the kernels: a
    longer prompt is taken whole too, in a form made for shorter ones.  The rest as gdr_decode, with
    q, k [N,qk_heads,Dk], v [N,H,Dv], g, beta [N,H].  An empty prompt leaves its slot as it is, or
    zero when fresh.  Tokens before the first prompt and after the last one have outputs 0."""
    if q.dim() != 3:
        raise ValueError("q must be [tokens, heads, Dk]")
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous() or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [sequences + 1] int32, contiguous")
    N = q.shape[0]
    max_len = min(plan.max_len, N) if max_len is None else max_len
    return _call(plan, 1, cu_seqlens.numel() - 1, N, max_len, q, k, v, g, beta, state, cu_seqlens, slots, fresh, o, stream)
