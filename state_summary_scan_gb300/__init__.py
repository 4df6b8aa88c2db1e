"""GB300-native chunkwise gated linear attention with per-segment affine
state summaries.

Layers:
  include/rm_cp.h          the C ABI (six compute calls + metadata builder)
  csrc/*.cu                sm_103a kernels behind it (librmcp.so, built in-tree)
  _capi                    ctypes binding, one Python function per C call
  api                      buffer allocation, call sequence, autograd adapter
  qk_rope, gdr_state,      the operators around the mixer: per-head norm with rotation, the gated
  gla_state, row_norm,     delta rule and linear attention on a pool of states (prefill, decoding),
  clip                     norms of rows with residual, gate and 8-bit outputs, gradient clipping
  workloads                seeded synthetic inputs (no method arithmetic)
"""
from . import _capi  # noqa: F401
from ._capi import RmCpError, ProblemSpec, load  # noqa: F401
from .api import (Plan, make_plan, plan_like, forward, backward,  # noqa: F401
                  chunkwise_gla, ChunkwiseGatedLinearAttention, GdrPlan, make_gdr_plan,
                  gdr_forward, gdr_backward, gated_delta_rule, GatedDeltaRule,
                  make_rope_table, qk_norm_rope, qk_norm_rope_backward, qk_norm_rope_train, QkNormRope,
                  GdrStatePlan, make_gdr_state_plan, make_gdr_state, gdr_decode, gdr_prefill,
                  GlaStatePlan, make_gla_state_plan, make_gla_state, gla_decode, gla_prefill,
                  rms_norm, rms_norm_quant, rms_norm_backward, rms_norm_train, RmsNorm,
                  ClipPlan, make_clip_plan, clip_grad_norm)
from .build import build as build_library  # noqa: F401

__all__ = ["RmCpError", "ProblemSpec", "load", "Plan", "make_plan", "plan_like", "forward",
           "backward", "chunkwise_gla", "ChunkwiseGatedLinearAttention", "GdrPlan", "make_gdr_plan",
           "gdr_forward", "gdr_backward", "gated_delta_rule", "GatedDeltaRule",
           "make_rope_table", "qk_norm_rope", "qk_norm_rope_backward", "qk_norm_rope_train", "QkNormRope",
           "GdrStatePlan", "make_gdr_state_plan", "make_gdr_state", "gdr_decode", "gdr_prefill",
           "GlaStatePlan", "make_gla_state_plan", "make_gla_state", "gla_decode", "gla_prefill",
           "rms_norm", "rms_norm_quant", "rms_norm_backward", "rms_norm_train", "RmsNorm",
           "ClipPlan", "make_clip_plan", "clip_grad_norm", "build_library"]
