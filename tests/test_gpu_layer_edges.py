"""Norm with rotation, the gated delta rule with a carried state, and clipping at the ends of what their
calls accept, against plain implementations in 64 bits (tolerances as in test_gpu_layer_ops.py)."""
import pytest
import torch

from state_summary_scan_gb300 import _capi as C
from state_summary_scan_gb300 import api
from test_gpu_layer_ops import BF16, F32, U, close, gds_check, gds_inputs, gds_ref, qkr_ref, rel2, rnd

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ the delta rule with a state

@pytest.mark.parametrize("lens,H,Hqk,Dk,Dv", [([1] * 5, 4, 2, 128, 128), ([1] * 3, 3, 3, 16, 40), ([4] * 3, 2, 1, 64, 72),
                                              ([9, 1, 0, 70], 2, 2, 128, 64), ([3, 1, 2], 2, 1, 32, 256)], ids=str)
def test_fp32_tokens_on_a_bf16_pool_call_by_call(lens, H, Hqk, Dk, Dv):
    """Each call's outputs are within fp32's tolerance of 64 bits from the states that it found: what the
    pool's rounding between two calls changes is not an error of the second."""
    S, state = len(lens), None
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    plan = api.make_gdr_state_plan(S, sum(lens), H, Dk, Dv, num_slots=S + 1, qk_heads=Hqk, max_len=max(lens), dtype=F32, state_dtype=BF16)
    tol = (max(lens) + Dk) * U
    for call in range(3):
        q, k, v, g, beta, first, slots = gds_inputs(lens, H, Hqk, Dk, Dv, F32, BF16, S + 1, seed=10 * call)
        state = first if state is None else state
        before = state.clone()
        o = api.gdr_prefill(plan, q, k, v, g, beta, state, cu, slots=slots.cuda())
        gds_check(lens, q, k, v, g, beta, before, state, o, slots, None, Dk ** -0.5, tol, tol)
        if len(set(lens)) == 1:  # the same call without cu_seqlens
            again = before.clone()
            o2 = api.gdr_decode(plan, *(x.unflatten(0, (S, lens[0])) for x in (q, k, v, g, beta)), again, slots=slots.cuda())
            assert torch.equal(o2.flatten(0, 1), o) and torch.equal(again, state)
