"""Linear attention on a pool of states against its recurrence in 64 bits.

Limits, element by element, from the formula's absolute sums (A for an output, B for a state element: the same
recurrence on |q|, |k|, |v|), with u = 2^-24 a rounding to fp32 and w = 2^-8 one to bf16 (half a step):
  recurrence  a token rounds the state twice and takes its decay with an error of up to 4 u, so the state is off by
              8 u a token; an output adds a sum of Dk terms: (8 n + Dk + 8) u A.
  chunks      P and S enter the outputs rounded to bf16: 2 w A (|P| and |S| are at most their absolute sums), which
              leaves out the second orders: 2.1 w A.  The state's sum of a chunk leaves 12 accumulations of up to 2 u
              each and its decays 8 u: 32 u B a chunk; V~ is exact to 2^-17 B for a bf16 pool.
  storing     bf16 outputs and states are rounded once more, by w of the value."""
import math

import pytest
import torch

from state_summary_scan_gb300 import _capi as C
from state_summary_scan_gb300 import api

pytestmark = pytest.mark.gpu
U, W = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


def plain(q, k, v, g, state, cu, slots, fresh, scale):
    """(o, pool) and their absolute sums (A, B) in 64 bits, on the host; q, k with the heads of v."""
    q, k, v, g, pool = (x.detach().double().cpu() for x in (q, k, v, g, state))
    r = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    o, A, B = torch.zeros_like(v), torch.zeros_like(v), pool.abs()
    for i, slot in enumerate(slots):
        if not 0 <= slot < pool.shape[0]:
            continue
        S = torch.zeros_like(pool[slot]) if fresh[i] else pool[slot].clone()
        T = S.abs()
        for t in range(cu[i], cu[i + 1]):
            a = g[t].exp()[:, None, None]
            S = a * S + k[t][:, :, None] * v[t][:, None, :]
            T = a * T + k[t].abs()[:, :, None] * v[t].abs()[:, None, :]
            o[t] = scale * torch.einsum("hkv,hk->hv", S, q[t])
            A[t] = abs(scale) * torch.einsum("hkv,hk->hv", T, q[t].abs())
        pool[slot], B[slot] = S, T
    return o, pool, A, B


def gates(kind, N, H, gen):
    if kind == "head":
        return -torch.logspace(math.log10(0.6), -4, H)
    if kind == "strong":  # some tokens forget nearly all, or all
        g = torch.nn.functional.logsigmoid(torch.randn(N, H, generator=gen) * 4)
        g[torch.rand(N, H, generator=gen) < 0.1] = -60.0
        g[torch.rand(N, H, generator=gen) < 0.05] = -math.inf
        return g
    return torch.nn.functional.logsigmoid(torch.randn(N, H, generator=gen) + 4)


def make(lens, H, Hqk, Dk, Dv, dtype, state_dtype, gate="token", seed=0, extra=(0, 0), slots_n=None):
    gen = torch.Generator().manual_seed(seed)
    N = sum(lens) + sum(extra)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    k = rnd(N, Hqk, Dk)
    x = dict(q=rnd(N, Hqk, Dk).to(dtype), k=(k / k.norm(dim=-1, keepdim=True)).to(dtype), v=rnd(N, H, Dv).to(dtype), g=gates(gate, N, H, gen))
    slots_n = slots_n or len(lens) + 2
    x["state"] = (0.5 * rnd(slots_n, H, Dk, Dv)).to(state_dtype)
    slots = torch.randperm(slots_n, generator=gen)[: len(lens)].to(torch.int32)
    fresh = (torch.arange(len(lens)) % 3 == 1).to(torch.uint8)
    cu = torch.tensor([0, *lens]).cumsum(0).to(torch.int32) + extra[0]
    return x, slots, fresh, cu


def check(o, state, want, lens, Dk, dtype, state_dtype, chunks):
    ro, rs, A, B = want
    n = max(lens)
    store = W if dtype == BF else 0.0
    far = (2.1 * W + 64 * U + 2.0 ** -16 if chunks else (8 * n + Dk + 8) * U) * A + store * ro.abs() + 1e-30
    err = (o.double().cpu() - ro).abs()
    assert bool((err <= far).all()), f"o: {float((err / far).max()):.2f} of its limit"
    if chunks:  # and in norm: P and S, and o itself, each rounded independently of one another (2^-8 / sqrt 3 each at most)
        assert float(err.norm()) <= 2.0 ** -8 * float(ro.norm()) * 1.05 + 1e-30
    acc = (32 * U * (n // 64 + 1) + (2.0 ** -17 if state_dtype == BF else 0) if chunks else 8 * n * U) + 4 * U
    far = acc * B + (W if state_dtype == BF else 0.0) * rs.abs() + 1e-30
    err = (state.double().cpu() - rs).abs()
    assert bool((err <= far).all()), f"state: {float((err / far).max()):.2f} of its limit"


def plan_of(x, lens, H, Hqk, Dk, Dv, **kw):
    return api.make_gla_state_plan(len(lens), x["q"].shape[0], H, Dk, Dv, num_slots=x["state"].shape[0], qk_heads=Hqk, max_len=max(lens),
                                   dtype=x["q"].dtype, state_dtype=x["state"].dtype, **kw)


def prefill(x, slots, fresh, cu, lens, H, Hqk, Dk, Dv, **kw):
    plan = plan_of(x, lens, H, Hqk, Dk, Dv, **kw)
    d = {n: t.cuda() for n, t in x.items()}
    o = api.gla_prefill(plan, d["q"], d["k"], d["v"], d["g"], d["state"], cu.cuda(), slots=slots.cuda(), fresh=fresh.cuda())
    return o, d["state"], plan


def reference(x, slots, fresh, cu, Dk):
    g = x["g"] if x["g"].dim() == 2 else x["g"].expand(x["q"].shape[0], -1)
    return plain(x["q"], x["k"], x["v"], g, x["state"], cu.tolist(), slots.tolist(), fresh.tolist(), Dk ** -0.5)


LENS = [0, 1, 47, 48, 63, 64, 65, 130, 200]


@pytest.mark.parametrize("dtype,state_dtype", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("H,Hqk,Dk,Dv,gate", [(2, 2, 64, 64, "token"), (2, 1, 128, 128, "head"), (2, 2, 128, 136, "strong"), (1, 1, 64, 8, "token"),
                                              (4, 2, 64, 40, "head"), (1, 1, 128, 256, "token"), (3, 3, 16, 24, "token"), (2, 1, 32, 64, "strong")])
def test_ragged_prompts(H, Hqk, Dk, Dv, gate, dtype, state_dtype):
    x, slots, fresh, cu = make(LENS, H, Hqk, Dk, Dv, dtype, state_dtype, gate)
    o, state, plan = prefill(x, slots, fresh, cu, LENS, H, Hqk, Dk, Dv)
    chunks = C.rm_cp_gla_state_path(plan.c) == 1
    assert chunks == (dtype == BF and Dk >= 64)  # (the longest has 200 tokens)
    check(o, state, reference(x, slots, fresh, cu, Dk), LENS, Dk, dtype, state_dtype, chunks)


@pytest.mark.parametrize("state_dtype", [F32, BF])
@pytest.mark.parametrize("H,Hqk,Dk,Dv,lens", [(2, 1, 64, 64, [1700]), (1, 1, 128, 128, [1025, 300, 1600]), (2, 2, 128, 200, [1281, 0, 64])])
def test_long_prompts_in_segments(H, Hqk, Dk, Dv, lens, state_dtype):
    x, slots, fresh, cu = make(lens, H, Hqk, Dk, Dv, BF, state_dtype, "head" if H == 2 else "token", seed=3)
    before = C.rm_cp_launch_count()
    o, state, _ = prefill(x, slots, fresh, cu, lens, H, Hqk, Dk, Dv)
    assert C.rm_cp_launch_count() - before == 3
    check(o, state, reference(x, slots, fresh, cu, Dk), lens, Dk, BF, state_dtype, True)


@pytest.mark.parametrize("dtype,state_dtype", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 9])
@pytest.mark.parametrize("H,Hqk,Dk,Dv,gate", [(2, 2, 128, 128, "token"), (4, 2, 16, 8, "head"), (2, 1, 32, 40, "strong"), (3, 3, 64, 264 - 8, "head")])
def test_decoding(H, Hqk, Dk, Dv, gate, n, dtype, state_dtype):
    S = 5
    x, slots, fresh, cu = make([n] * S, H, Hqk, Dk, Dv, dtype, state_dtype, gate, seed=n)
    slots[2] = -1  # padding
    plan = plan_of(x, [n] * S, H, Hqk, Dk, Dv)
    d = {m: t.cuda() for m, t in x.items()}
    split = lambda t: t.unflatten(0, (S, n)) if t.dim() > 1 else t  # noqa: E731
    o = api.gla_decode(plan, split(d["q"]), split(d["k"]), split(d["v"]), split(d["g"]), d["state"], slots=slots.cuda(), fresh=fresh.cuda())
    check(o.flatten(0, 1), d["state"], reference(x, slots, fresh, cu, Dk), [n], Dk, dtype, state_dtype, False)


@pytest.mark.parametrize("dtype,Dk,Dv,T,recurrent", [(BF, 128, 128, 2048, False), (BF, 64, 64, 2048, False), (BF, 32, 48, 2048, False), (BF, 64, 64, 31, False),
                                                     (BF, 64, 64, 2048, True), (F32, 64, 64, 2048, False), (F32, 64, 64, 1024, True), (F32, 128, 128, 8, False)])
def test_slow_decays_lose_no_bits(dtype, Dk, Dv, T, recurrent):
    """One decay near 1 for every token.  A decay rounded to fp32, or sums that are cut off, would be off the same way each
    time: some T u of the state.  Roundings to nearest add up like sqrt(T), of a memory of 1000 tokens at most: three of them
    a token stay within 3 sqrt(min(T, 1000)) u of its norm."""
    x, slots, fresh, cu = make([T], 2, 2, Dk, Dv, dtype, F32, seed=11)
    x["g"] = torch.tensor([-1.0e-3, -1.7e-3])
    _, state, _ = prefill(x, slots, fresh, cu, [T], 2, 2, Dk, Dv, recurrent=recurrent)
    want = reference(x, slots, fresh, cu, Dk)[1][slots[0]]
    assert float((state[slots[0]].double().cpu() - want).norm() / want.norm()) <= 3 * math.sqrt(min(T, 1000)) * U
