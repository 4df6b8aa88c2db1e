"""Prompts cut into segments of many chunks, with a gate for each token: every ring of the walks is used several times over, in
segments with outputs and in those without.  And the outputs of prompts that are longer than a bound of a few tokens.

The limits are those of test_gpu_gla_state.py, against the recurrence in 64 bits in blocks (blocks())."""
import pytest
import torch
from test_gpu_gla_state import BF, F32, check, make, plain, plan_of, reference

from state_summary_scan_gb300 import _capi as C
from state_summary_scan_gb300 import api

pytestmark = pytest.mark.gpu


def blocks(x, slots, fresh, cu, scale, size=64):
    """plain() of test_gpu_gla_state.py on the GPU, `size` tokens at a time: with b the running sum of a block's gates and S the
    state before it, o_t = e^b_t S^T q_t + sum over r <= t of e^(b_t - b_r) (q_t.k_r) v_r."""
    q, k, v, pool = (x[n].double().cuda() for n in ("q", "k", "v", "state"))
    g = x["g"].double().cuda().clamp(min=-1000.0)  # e^-1000 is 0
    r = v.shape[1] // q.shape[1]
    q, k, v = q.repeat_interleave(r, 1).transpose(0, 1), k.repeat_interleave(r, 1).transpose(0, 1), v.transpose(0, 1)
    g = g.t() if g.dim() == 2 else g[:, None].expand(-1, q.shape[1])
    o, A, B = torch.zeros_like(v), torch.zeros_like(v), pool.abs()
    for i, slot in enumerate(slots.tolist()):
        S = torch.zeros_like(pool[slot]) if fresh[i] else pool[slot].clone()
        T = S.abs()
        for t in range(int(cu[i]), int(cu[i + 1]), size):
            at = slice(t, min(t + size, int(cu[i + 1])))
            b = g[:, at].cumsum(1)
            fade, to_end, end = (b[:, :, None] - b[:, None]).tril().exp().tril(), (b[:, -1:] - b).exp()[..., None], b[:, -1].exp()[:, None, None]
            for qq, kk, vv, state, out in ((q[:, at], k[:, at], v[:, at], S, o), (q[:, at].abs(), k[:, at].abs(), v[:, at].abs(), T, A)):
                out[:, at] = scale * (b.exp()[..., None] * (qq @ state) + ((qq @ kk.mT) * fade) @ vv)
                state.copy_(end * state + (kk * to_end).mT @ vv)
        pool[slot], B[slot] = S, T
    return o.transpose(0, 1).cpu(), pool.cpu(), A.transpose(0, 1).cpu(), B.cpu()


@pytest.mark.parametrize("gate", ["token", "strong", "head"])
def test_blocks_are_the_recurrence(gate):
    x, slots, fresh, cu = make([130, 0, 63, 64], 4, 2, 16, 24, BF, F32, gate, seed=1)
    g = x["g"] if x["g"].dim() == 2 else x["g"].expand(x["q"].shape[0], -1)
    want = plain(x["q"], x["k"], x["v"], g, x["state"], cu.tolist(), slots.tolist(), fresh.tolist(), 0.25)
    for got, w, size in zip(blocks(x, slots, fresh, cu, 0.25), want, (want[2], want[3]) * 2):
        assert bool(((got - w).abs() <= 1e-10 * size + 1e-30).all())


@pytest.mark.parametrize("state_dtype", [F32, BF])
@pytest.mark.parametrize("H,Hqk,Dk,Dv,lens,gate", [
    (16, 16, 128, 128, [8192], "token"),  # after the first segment nine of 14 chunks
    (16, 8, 128, 128, [4096], "token"),  # nine of 7
    (32, 32, 128, 128, [2040], "strong"),  # four of 7
    (4, 4, 64, 64, [8190], "token"),  # 25 of 5
    (2, 2, 64, 64, [4096, 4095, 2500, 0, 1, 449, 3000, 64], "token"),  # nine of 7 of the longest
    (2, 1, 128, 200, [4000, 1793, 1792, 640], "strong"),  # eight of 7
])
def test_long_segments_with_a_gate_for_each_token(H, Hqk, Dk, Dv, lens, gate, state_dtype):
    x, slots, fresh, cu = make(lens, H, Hqk, Dk, Dv, BF, state_dtype, gate, seed=len(lens) + H)
    plan = plan_of(x, lens, H, Hqk, Dk, Dv)
    d = {n: t.cuda() for n, t in x.items()}
    at = (cu.cuda(), slots.cuda(), fresh.cuda())
    before = C.rm_cp_launch_count()

    def call():
        state = d["state"].clone()
        return api.gla_prefill(plan, d["q"], d["k"], d["v"], d["g"], state, at[0], slots=at[1], fresh=at[2]), state

    o, state = call()
    assert C.rm_cp_launch_count() - before == 3  # it was cut
    check(o, state, blocks(x, slots, fresh, cu, Dk ** -0.5), lens, Dk, BF, state_dtype, True)
    # the same bits whatever the groups of a walk wait for: tokens that come late, beside copies on another stream
    side, big = torch.cuda.Stream(), torch.empty(2, 1 << 28, dtype=torch.uint8, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(30):
            big[0].copy_(big[1])
    again = [call() for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(p, o) and torch.equal(s, state) for p, s in again)
    assert C.rm_cp_device_status(torch.zeros(1, dtype=torch.int32, device="cuda")) == 0  # no wait ran out


@pytest.mark.parametrize("Dk,Dv", [(128, 64), (64, 40), (16, 24)])
@pytest.mark.parametrize("max_len", [1, 2, 4])
def test_outputs_of_prompts_longer_than_a_bound_of_a_few_tokens(max_len, Dk, Dv):
    """A bf16 pool is then rounded every four tokens, by w = 2^-8 of it, and the rounded states are what the next tokens see.  Every
    head's decay is e^-0.6 or less: of a rounding e^-2.4 is left four tokens on, 1 / (1 - e^-2.4) = 1.1 of them in all."""
    lens = [650, 5, 0, 66, 1]
    x, slots, fresh, cu = make(lens, 2, 1, Dk, Dv, BF, BF, "head", seed=4)
    x["g"] = torch.tensor([-0.6, -0.9])
    plan = api.make_gla_state_plan(5, sum(lens), 2, Dk, Dv, num_slots=7, qk_heads=1, state_dtype=BF)
    d = {n: t.cuda() for n, t in x.items()}
    o = api.gla_prefill(plan, d["q"], d["k"], d["v"], d["g"], d["state"], cu.cuda(), slots=slots.cuda(), fresh=fresh.cuda(), max_len=max_len)
    want, pool, A, B = reference(x, slots, fresh, cu, Dk)
    u, w = 2.0 ** -24, 2.0 ** -8
    assert bool(((o.double().cpu() - want).abs() <= (1.1 * w + (8 * 650 + Dk + 8) * u) * A + w * want.abs() + 1e-30).all())
    assert bool(((d["state"].double().cpu() - pool).abs() <= (1.1 * w + (8 * 650 + 4) * u) * B + w * pool.abs() + 1e-30).all())
