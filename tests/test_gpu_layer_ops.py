"""Per-head norm with rotation, the gated delta rule with a carried state, and gradient clipping,
against plain implementations in 64 bits.

Tolerances.  fp32: u = 2^-24 a rounding.  A head row is at most 256 squares (summed by lanes: 8 in
a lane, 5 levels) and about ten more roundings, so an element is within 32 u of the largest one:
2e-6.  bf16 results (8 significant bits) add half a unit in the last place: at most
2^-8 of the element itself.  A weight's
gradient adds N products in a fixed tree, 2^-24 (N_thread + levels) of the sum of their magnitudes.
The recurrence in fp32 makes (Dk + 8) roundings a token on values that do not grow:
n (Dk + 8) u of the largest value at worst, about its square root in practice; (n + Dk) u is used.
"""
import math

import pytest
import torch

from state_summary_scan_gb300 import _capi as C
from state_summary_scan_gb300 import api

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def rnd(*s, seed=0, dtype=F32):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(*s, generator=g, device="cuda").to(dtype)


def close(got, want, tol, dtype, what):
    """|got - want| <= tol max|want| (+ the rounding of a bf16 result)."""
    got, want = got.double(), want.double()
    lim = tol * float(want.abs().max()) + (want.abs() * 2.0 ** -8 if dtype == BF16 else 0.0) + 1e-40
    bad = (got - want).abs() - lim
    assert not torch.isnan(got).any(), what
    assert float(bad.max()) <= 0, (what, float((got - want).abs().max()), float(want.abs().max()))


# ------------------------------------------------------------------ norm and rotation

def qkr_ref(x, w, table, pos, norm, eps, inter):
    """One of q, k in fp64: x [B,T,H,D], table [P,2,R/2], pos [B,T]."""
    y = x
    if norm == "rms":
        y = x * (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    elif norm == "l2":
        y = x * (x.pow(2).sum(-1, keepdim=True) + eps).rsqrt()
    y = y if w is None else y * w
    if table is None:
        return y
    R = 2 * table.shape[2]
    c, s = table[pos][:, :, None].unbind(3)
    a, b = (y[..., 0:R:2], y[..., 1:R:2]) if inter else (y[..., : R // 2], y[..., R // 2: R])
    a, b = a * c - b * s, b * c + a * s
    both = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([both, y[..., R:]], -1)


QKR = [
    # B, T, Hq, Hk, D, R, norm, weights, interleaved, dtype, fused, positions
    (1, 1, 1, 1, 8, 8, "rms", True, False, F32, False, None),
    (2, 5, 4, 2, 128, 128, "rms", True, False, BF16, False, "BT"),
    (2, 5, 4, 2, 128, 128, "rms", True, True, F32, True, "T64"),
    (1, 700, 16, 16, 128, 128, "rms", True, False, BF16, True, None),
    (1, 1300, 5, 3, 64, 16, "l2", False, True, BF16, True, "BT64"),
    (3, 7, 3, 1, 80, 40, "l2", True, False, F32, False, "BT"),     # pairs that straddle lanes
    (2, 3, 2, 2, 96, 20, "rms", False, True, F32, True, "T"),      # a partly rotated lane
    (1, 9, 2, 1, 256, 256, "none", True, False, BF16, False, "T"),
    (1, 4, 7, 7, 32, 2, "none", False, False, F32, False, "BT"),
    (2, 33, 9, 2, 24, 0, "rms", True, False, F32, True, None),
    (1, 2, 33, 1, 248, 248, "l2", True, False, BF16, False, "T64"),
]


def qkr_inputs(case, seed=0):
    B, T, Hq, Hk, D, R, norm, weights, inter, dtype, fused, pos = case
    if fused:
        x = (2 * rnd(B, T, (Hq + 2 * Hk) * D, seed=seed)).to(dtype)
        q, k = x[..., : Hq * D].unflatten(-1, (Hq, D)), x[..., Hq * D: (Hq + Hk) * D].unflatten(-1, (Hk, D))
    else:
        q, k = rnd(B, T, Hq, D, seed=seed, dtype=dtype), rnd(B, T, Hk, D, seed=seed + 1, dtype=dtype)
    table = api.make_rope_table(2000, R) if R else None
    g = torch.Generator("cuda").manual_seed(seed + 2)
    p = None
    if pos:
        shape = (B, T) if pos.startswith("BT") else (T,)
        p = torch.randint(0, 2000, shape, generator=g, device="cuda", dtype=torch.int64 if pos.endswith("64") else torch.int32)
    w = (1 + 0.3 * rnd(D, seed=seed + 3), 1 + 0.3 * rnd(D, seed=seed + 4)) if weights else (None, None)
    how = dict(table=table, positions=p, q_weight=w[0], k_weight=w[1], norm=norm, eps=1e-5, interleaved=inter)
    full = (torch.arange(T, device="cuda") if p is None else p.long()).expand(B, T)
    return q, k, how, full


@pytest.mark.parametrize("case", QKR, ids=str)
def test_qkr_against_64_bits(case):
    q, k, how, pos = qkr_inputs(case)
    dtype, tol = q.dtype, 32 * U
    t64 = None if how["table"] is None else how["table"].double()
    before = q.clone(), k.clone()
    got = api.qk_norm_rope(q, k, **how)
    dy = [rnd(*x.shape, seed=9 + i, dtype=dtype) for i, x in enumerate((q, k))]
    back = api.qk_norm_rope_backward(q, k, *dy, **how)
    assert torch.equal(q, before[0]) and torch.equal(k, before[1])
    for i, (x, w) in enumerate(((q, how["q_weight"]), (k, how["k_weight"]))):
        x64 = x.double().requires_grad_(True)
        w64 = None if w is None else w.double().requires_grad_(True)
        y = qkr_ref(x64, w64, t64, pos, how["norm"], how["eps"], how["interleaved"])
        close(got[i], y.detach(), tol, dtype, f"output {i}")
        want = torch.autograd.grad(y, [x64] + ([] if w is None else [w64]), dy[i].double())
        close(back[i], want[0], 2 * tol, dtype, f"gradient {i}")
        if w is None:
            assert back[2 + i] is None
        else:
            # rows a thread adds, then at most 2^12 partial sums in levels
            n = x.numel() // x.shape[-1]
            scale = float((dy[i].double().abs() * 4).sum((0, 1, 2)).max())
            assert float((back[2 + i].double() - want[1]).abs().max()) <= (32 + n / 64) * U * scale, f"weight {i}"


def test_qkr_gradient_against_differences():
    case = (1, 3, 2, 2, 64, 32, "rms", True, False, F32, False, "T")
    q, k, how, _ = qkr_inputs(case)
    dy = [rnd(*x.shape, seed=3 + i) for i, x in enumerate((q, k))]
    back = api.qk_norm_rope_backward(q, k, *dy, **how)

    def loss(q, k, wq, wk):
        y = api.qk_norm_rope(q, k, **{**how, "q_weight": wq, "k_weight": wk})
        return sum(float((a.double() * b.double()).sum()) for a, b in zip(y, dy))

    at = [q, k, how["q_weight"], how["k_weight"]]
    for i in range(4):
        d, h = rnd(*at[i].shape, seed=20 + i), 2.0 ** -7
        up, dn = list(at), list(at)
        up[i], dn[i] = at[i] + h * d, at[i] - h * d
        diff = (loss(*up) - loss(*dn)) / (2 * h)
        want = float((back[i].double() * d.double()).sum())
        # truncation h^2 / 6 of third derivatives (rows of unit size: at most about 10 |dy| |d|),
        # roundings 16 u of 384 outputs over h
        n = math.sqrt(d.numel())
        assert abs(diff - want) <= 10 * h * h * n + 16 * U * 384 / h, (i, diff, want)


def test_qkr_rows_of_zeros_and_bad_positions():
    q, k = rnd(1, 4, 2, 64), rnd(1, 4, 1, 64, seed=1)
    q[0, 1] = 0
    q[0, 2, 0, 5] = float("nan")
    table = api.make_rope_table(10, 32)
    pos = torch.tensor([3, 4, 5, 10], device="cuda", dtype=torch.int32)  # the last lies outside
    y, z = api.qk_norm_rope(q, k, table, pos, norm="l2", eps=1e-6)
    assert torch.equal(y[0, 1], torch.zeros_like(y[0, 1]))
    assert torch.isnan(y[0, 2, 0]).all() and not torch.isnan(y[0, 2, 1]).any()
    for x in (y, z):
        assert torch.isnan(x[0, 3, :, :32]).all() and not torch.isnan(x[0, 3, :, 32:]).any()
    neg = torch.tensor([-1, -(1 << 31), 1, 2], device="cuda", dtype=torch.int32)
    y, _ = api.qk_norm_rope(k, k, table, neg)
    assert torch.isnan(y[0, :2, :, :32]).all() and not torch.isnan(y[0, 2:]).any()
    dq, dk, _, _ = api.qk_norm_rope_backward(q, k, torch.ones_like(q), torch.ones_like(k), table, pos, norm="l2", eps=1e-6)
    assert torch.isfinite(dq[0, 1]).all()  # the gradient at a zero row: 1 / sqrt(eps)


def test_qkr_single_tokens_equal_the_prompt():
    case = (2, 19, 4, 2, 128, 64, "rms", True, False, BF16, True, "BT")
    q, k, how, _ = qkr_inputs(case)
    y, z = api.qk_norm_rope(q, k, **how)
    for t in range(19):
        one = {**how, "positions": how["positions"][:, t: t + 1].contiguous()}
        a, b = api.qk_norm_rope(q[:, t: t + 1], k[:, t: t + 1], **one)
        assert torch.equal(a, y[:, t: t + 1]) and torch.equal(b, z[:, t: t + 1])


def test_qkr_adapter_stream_and_empty():
    case = (2, 65, 4, 4, 64, 64, "rms", True, True, F32, False, "BT")
    q, k, how, _ = qkr_inputs(case)
    leaves = [x.clone().requires_grad_(True) for x in (q, k, how["q_weight"], how["k_weight"])]
    y, z = api.qk_norm_rope_train(leaves[0], leaves[1], how["table"], how["positions"], leaves[2], leaves[3], how["norm"], how["eps"], True)
    dy = rnd(*y.shape, seed=4), rnd(*z.shape, seed=5)
    got = torch.autograd.grad([y, z], leaves, dy)
    want = api.qk_norm_rope_backward(q, k, *dy, **how)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(q), torch.empty_like(k)
    api.qk_norm_rope(q, k, **how, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out[0], y.detach()) and torch.equal(out[1], z.detach())
    e = torch.empty(2, 0, 4, 64, device="cuda")
    y, z = api.qk_norm_rope(e, e, how["table"])
    assert y.shape == e.shape
    dq, dk, dwq, dwk = api.qk_norm_rope_backward(e, e, e, e, how["table"], q_weight=how["q_weight"], k_weight=how["k_weight"])
    assert not dwq.any() and not dwk.any()


def test_qkr_refuses():
    q = rnd(2, 3, 4, 64)
    t = api.make_rope_table(8, 64)
    for bad in (dict(norm="other"), dict(positions=torch.zeros(5, device="cuda", dtype=torch.int32)), dict(positions=torch.zeros(3, device="cuda")),
                dict(q_weight=torch.ones(32, device="cuda")), dict(k_weight=torch.ones(64, device="cuda", dtype=BF16)), dict(table=t[:, :1])):
        with pytest.raises(ValueError):
            api.qk_norm_rope(q, q, **{**dict(table=t), **bad})
    with pytest.raises(ValueError):
        api.qk_norm_rope(q, q.to(BF16), t)
    with pytest.raises(ValueError):
        api.qk_norm_rope(q.transpose(2, 3), q.transpose(2, 3), t)
    with pytest.raises(C.RmCpError) as e:
        api.qk_norm_rope(q, q, api.make_rope_table(8, 128))  # more than the head
    assert e.value.status == 1
    with pytest.raises(C.RmCpError) as e:
        x = rnd(2, 3, 4 * 64 + 1)[..., 1:].unflatten(-1, (4, 64))
        api.qk_norm_rope(x, x, t)
    assert e.value.status == 3


# ------------------------------------------------------------------ the delta rule with a state

def gds_ref(q, k, v, g, beta, S, scale):
    """One sequence, token by token in fp64: q, k [n,Hqk,Dk], v [n,H,Dv], S [H,Dk,Dv]."""
    r = v.shape[1] // q.shape[1]
    q, k = q.double().repeat_interleave(r, 1), k.double().repeat_interleave(r, 1)
    v, g, beta, S = v.double(), g.double(), beta.double(), S.double()
    o = []
    for t in range(q.shape[0]):
        S = S * g[t].exp()[:, None, None]
        d = beta[t][:, None] * (v[t] - torch.einsum("hk,hkv->hv", k[t], S))
        S = S + k[t][:, :, None] * d[:, None]
        o.append(scale * torch.einsum("hk,hkv->hv", q[t], S))
    return (torch.stack(o) if o else v), S


def gds_inputs(lens, H, Hqk, Dk, Dv, dtype, state_dtype, slots_n, seed=0, fused=False):
    N = sum(lens)
    if fused:  # q, k, v of one projection
        F = 2 * Hqk * Dk + H * Dv
        x = rnd(N, F, seed=seed, dtype=dtype)
        x[:, Hqk * Dk: 2 * Hqk * Dk] *= Dk ** -0.5
        q, k, v = (y.unflatten(-1, (h, -1)) for y, h in zip(x.split([Hqk * Dk, Hqk * Dk, H * Dv], -1), (Hqk, Hqk, H)))
    else:
        q, k, v = rnd(N, Hqk, Dk, seed=seed, dtype=dtype), rnd(N, Hqk, Dk, seed=seed + 1), rnd(N, H, Dv, seed=seed + 2, dtype=dtype)
        k = (k / k.norm(dim=-1, keepdim=True)).to(dtype)
    g = torch.nn.functional.logsigmoid(rnd(N, H, seed=seed + 3) + 3)
    beta = torch.sigmoid(rnd(N, H, seed=seed + 4))
    state = rnd(slots_n, H, Dk, Dv, seed=seed + 5, dtype=state_dtype)
    slots = torch.randperm(slots_n, generator=torch.Generator().manual_seed(seed))[: len(lens)].to(torch.int32)
    return q, k, v, g, beta, state, slots


def gds_check(lens, q, k, v, g, beta, before, after, o, slots, fresh, scale, tol, otol):
    at, touched = 0, set()
    for i, n in enumerate(lens):
        s = slice(at, at + n)
        at += n
        j = int(slots[i])
        if not 0 <= j < before.shape[0]:
            assert not o[s].any()
            continue
        touched.add(j)
        S0 = torch.zeros_like(before[j]) if fresh is not None and int(fresh[i]) else before[j]
        want_o, want_S = gds_ref(q[s], k[s], v[s], g[s], beta[s], S0, scale)
        if n:
            close(o[s], want_o, otol, o.dtype, f"o of sequence {i}")
        close(after[j], want_S, tol, after.dtype, f"state of sequence {i}")
    for j in set(range(before.shape[0])) - touched:
        assert torch.equal(after[j], before[j]), f"slot {j}"


DECODE = [  # S, n, H, Hqk, Dk, Dv, dtype, state dtype, fused
    (1, 1, 1, 1, 16, 8, F32, F32, False),
    (3, 1, 4, 2, 64, 64, BF16, F32, True),
    (5, 4, 6, 3, 128, 256, BF16, BF16, False),
    (2, 7, 2, 2, 32, 40, F32, F32, False),
    (4, 2, 3, 1, 128, 24, F32, BF16, True),
    (9, 1, 16, 16, 128, 128, BF16, F32, True),
    (2, 33, 2, 1, 64, 128, BF16, F32, False),
    (5, 1, 4, 2, 128, 136, BF16, BF16, True),
    (3, 3, 3, 3, 16, 40, BF16, BF16, False),
    (4, 5, 4, 4, 128, 8, BF16, BF16, True),
    (1, 39, 2, 1, 32, 256, BF16, BF16, False),
    (3, 4, 2, 2, 64, 72, BF16, F32, True),
]


@pytest.mark.parametrize("case", DECODE, ids=str)
@pytest.mark.parametrize("fresh", [False, True])
def test_gdr_decode_against_64_bits(case, fresh):
    S, n, H, Hqk, Dk, Dv, dtype, sdt, fused = case
    q, k, v, g, beta, state, slots = gds_inputs([n] * S, H, Hqk, Dk, Dv, dtype, sdt, S + 2, fused=fused)
    if S > 2:
        slots[1] = -1      # padding sequences
        slots[2] = S + 2
    fr = (torch.arange(S) % 2 == 0).to(torch.uint8) if fresh else None
    plan = api.make_gdr_state_plan(S, S * n, H, Dk, Dv, num_slots=S + 2, qk_heads=Hqk, dtype=dtype, state_dtype=sdt)
    before = state.clone()
    lead = [x.unflatten(0, (S, n)) for x in (q, k, v, g, beta)]
    o = api.gdr_decode(plan, *lead, state, slots=slots.cuda(), fresh=None if fr is None else fr.cuda())
    tol = (n + Dk) * U
    gds_check([n] * S, q, k, v, g, beta, before, state, o.flatten(0, 1), slots, fr, Dk ** -0.5, tol, tol)


PREFILL = [  # lens, H, Hqk, Dk, Dv, dtype, state dtype
    ([1], 1, 1, 16, 8, F32, F32),
    ([0, 5, 1, 63, 130, 0], 4, 2, 32, 40, F32, F32),
    ([64, 65, 200], 2, 2, 128, 128, F32, F32),
    ([17, 0, 100], 3, 1, 32, 72, BF16, F32),
    ([1, 4, 5, 0, 39, 2, 8], 4, 2, 128, 72, BF16, F32),
    ([0, 7, 0, 38], 2, 1, 64, 256, BF16, BF16),
    ([2, 3, 4, 1, 0], 3, 3, 128, 136, BF16, BF16),
    ([13, 29], 2, 2, 16, 40, BF16, F32),
]


@pytest.mark.parametrize("case", PREFILL, ids=str)
def test_gdr_prefill_token_recurrence_against_64_bits(case):
    lens, H, Hqk, Dk, Dv, dtype, sdt = case
    S = len(lens)
    q, k, v, g, beta, state, slots = gds_inputs(lens, H, Hqk, Dk, Dv, dtype, sdt, S + 1)
    fr = (torch.arange(S) % 3 == 0).to(torch.uint8)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    plan = api.make_gdr_state_plan(S, sum(lens), H, Dk, Dv, num_slots=S + 1, qk_heads=Hqk, max_len=max(lens), dtype=dtype,
                                   state_dtype=sdt)
    assert C.rm_gdr_state_path(plan.c) == 0
    before = state.clone()
    o = api.gdr_prefill(plan, q, k, v, g, beta, state, cu, slots=slots.cuda(), fresh=fr.cuda())
    tol = (max(lens) + Dk) * U
    gds_check(lens, q, k, v, g, beta, before, state, o, slots, fr, Dk ** -0.5, tol, tol)


# In chunks on the tensor cores: S, W = T (K o gam) and P = mask(Q K^T) are rounded to bf16 once
# (2^-8 at worst, 1.7e-3 in norm), o itself once more: four independent roundings in norm, at most
# 3.4e-3 < 2^-8 for o; the state sees only those of S and W, through W S, which the unit keys keep
# small beside T V: 2e-3 is the norm of one whole rounding of it.
CHUNKED = [  # lens, H, Hqk, Dk, Dv, state dtype, fused
    ([64], 1, 1, 128, 128, F32, False),
    ([128, 64], 2, 2, 64, 64, F32, False),
    ([100], 1, 1, 128, 64, BF16, True),
    ([0, 5, 1, 63, 130, 64, 0, 65], 4, 2, 128, 128, F32, False),
    ([333, 1, 200], 3, 1, 64, 200, BF16, True),
    ([1000, 77], 2, 1, 128, 256, F32, True),
    ([511, 513], 2, 2, 64, 128, BF16, False),
]


def rel2(got, want):
    return float((got.double() - want.double()).norm() / (want.double().norm() + 1e-300))


@pytest.mark.parametrize("case", CHUNKED, ids=str)
def test_gdr_prefill_in_chunks_against_64_bits(case):
    lens, H, Hqk, Dk, Dv, sdt, fused = case
    S = len(lens)
    q, k, v, g, beta, state, slots = gds_inputs(lens, H, Hqk, Dk, Dv, BF16, sdt, S + 1, fused=fused)
    fr = (torch.arange(S) % 2 == 1).to(torch.uint8)
    if S > 4:
        slots[3] = S + 7  # a padding sequence
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    plan = api.make_gdr_state_plan(S, sum(lens), H, Dk, Dv, num_slots=S + 1, qk_heads=Hqk, state_dtype=sdt)
    assert C.rm_gdr_state_path(plan.c) == 1
    before = state.clone()
    o = api.gdr_prefill(plan, q, k, v, g, beta, state, cu, slots=slots.cuda(), fresh=fr.cuda())
    scratch = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert C.rm_cp_device_status(scratch) == 0
    at, touched = 0, set()
    for i, n in enumerate(lens):
        s, j = slice(at, at + n), int(slots[i])
        at += n
        if not 0 <= j < S + 1:
            assert not o[s].any()
            continue
        touched.add(j)
        S0 = torch.zeros_like(before[j]) if int(fr[i]) else before[j]
        want_o, want_S = gds_ref(q[s], k[s], v[s], g[s], beta[s], S0, Dk ** -0.5)
        if n:
            assert rel2(o[s], want_o) <= 2.0 ** -8, (i, rel2(o[s], want_o))
            close(o[s], want_o, 2e-2, BF16, f"o of sequence {i}")
            assert rel2(state[j], want_S) <= 2e-3 + (2.0 ** -8 if sdt == BF16 else 0), (i, rel2(state[j], want_S))
        else:
            assert torch.equal(state[j], S0)
    for j in set(range(S + 1)) - touched:
        assert torch.equal(state[j], before[j])


@pytest.mark.parametrize("Dk,Dv,sdt,strong", [(128, 128, F32, False), (128, 136, BF16, False), (64, 64, F32, True), (64, 256, F32, False)])
def test_gdr_prefill_in_segments_against_64_bits(Dk, Dv, sdt, strong):
    """Few heads and long prompts: the walk is cut into segments whose maps are composed."""
    lens, H, Hqk = [4100, 0, 130, 2500, 3000], 2, 1
    S = len(lens)
    q, k, v, g, beta, state, slots = gds_inputs(lens, H, Hqk, Dk, Dv, BF16, sdt, S + 1, seed=4)
    if strong:  # chunks of strong decay among weak ones, and forgotten states
        g[300:420, 0] = -3.0
        g[900] = -float("inf")
        g[2000:2300, 1] *= 40
        g[5000:5070, 0] = -4.0
    fr = torch.tensor([0, 1, 0, 1, 0], dtype=torch.uint8)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    plan = api.make_gdr_state_plan(S, sum(lens), H, Dk, Dv, num_slots=S + 1, qk_heads=Hqk, state_dtype=sdt)
    before, n0 = state.clone(), C.rm_cp_launch_count()
    o = api.gdr_prefill(plan, q, k, v, g, beta, state, cu, slots=slots.cuda(), fresh=fr.cuda(), max_len=4100)
    assert C.rm_cp_launch_count() - n0 == 4  # factors, first walk, composition, second walk
    assert C.rm_cp_device_status(torch.zeros(4, dtype=torch.int32, device="cuda")) == 0
    at = 0
    for i, n in enumerate(lens):
        s, j = slice(at, at + n), int(slots[i])
        at += n
        S0 = torch.zeros_like(before[j]) if int(fr[i]) else before[j]
        want_o, want_S = gds_ref(q[s], k[s], v[s], g[s], beta[s], S0, Dk ** -0.5)
        if n:
            assert rel2(o[s], want_o) <= 2.0 ** -8, (i, rel2(o[s], want_o))
            assert rel2(state[j], want_S) <= 2e-3 + (2.0 ** -8 if sdt == BF16 else 0), (i, rel2(state[j], want_S))
        else:
            assert torch.equal(state[j], S0)
    idle = (set(range(S + 1)) - set(slots.tolist())).pop()
    assert torch.equal(state[idle], before[idle])


def test_gdr_prefill_in_chunks_keeps_nan_and_resets_apart():
    """A NaN key or value stays in its own sequence, on both sides of a shared tile; g = -inf
    forgets the state; the same call twice gives the same bits."""
    lens, H, D = [70, 50, 90], 2, 128
    q, k, v, g, beta, state, slots = gds_inputs(lens, H, H, D, D, BF16, F32, 3, seed=5)
    v[75, 0, 3] = float("nan")
    k[100, 1, 0] = float("nan")
    q[80] = float("inf")
    g[30] = -float("inf")
    g[120 + 64] = -1e30
    g[120 + 10] = -500.0
    plan = api.make_gdr_state_plan(3, 210, H, D, D)
    cu = torch.tensor([0, 70, 120, 210], dtype=torch.int32, device="cuda")
    before = state.clone()
    o = api.gdr_prefill(plan, q, k, v, g, beta, state, cu, slots=slots.cuda())
    for i, s in ((0, slice(0, 70)), (2, slice(120, 210))):
        j = int(slots[i])
        want_o, want_S = gds_ref(q[s], k[s], v[s], g[s], beta[s], before[j], D ** -0.5)
        assert rel2(o[s], want_o) <= 2.0 ** -8 and rel2(state[j], want_S) <= 2e-3
    again = before.clone()
    o2 = api.gdr_prefill(plan, q, k, v, g, beta, again, cu, slots=slots.cuda())
    for i, s in ((0, slice(0, 70)), (2, slice(120, 210))):
        assert torch.equal(o2[s], o[s]) and torch.equal(again[int(slots[i])], state[int(slots[i])])


def test_gdr_prefill_in_parts_continues_the_state():
    """A prompt in two calls, the second from the state of the first, against the whole."""
    T, H, D, cut = 300, 2, 128, 130
    q, k, v, g, beta, state, _ = gds_inputs([T], H, H, D, D, BF16, F32, 1, seed=9)
    plan = api.make_gdr_state_plan(1, T, H, D, D)
    whole, parts = state.clone(), state.clone()
    want = api.gdr_prefill(plan, q, k, v, g, beta, whole, torch.tensor([0, T], dtype=torch.int32, device="cuda"))
    got = []
    for a, b in ((0, cut), (cut, T)):
        cu = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        got.append(api.gdr_prefill(plan, *(x[a:b] for x in (q, k, v, g, beta)), parts, cu))
    assert rel2(torch.cat(got), want) <= 2.0 ** -8 and rel2(parts, whole) <= 2e-3


def test_gdr_prefill_then_decode_equals_the_training_op():
    """The state handed over continues the recurrence that the training calls compute."""
    T, H, D = 96, 2, 32
    q, k, v, g, beta, _, _ = gds_inputs([T], H, H, D, D, F32, F32, 1, seed=7)
    train = api.make_gdr_plan(1, T, H, D, D, 3)
    want = api.gdr_forward(train, *(x[None].contiguous() for x in (q, k, v, g, beta)))[0]
    plan = api.make_gdr_state_plan(1, T, H, D, D, dtype=F32)
    state = api.make_gdr_state(plan)
    cut = 70
    cu = torch.tensor([0, cut], dtype=torch.int32, device="cuda")
    got = [api.gdr_prefill(plan, *(x[:cut] for x in (q, k, v, g, beta)), state, cu)]
    for t in range(cut, T):
        got.append(api.gdr_decode(plan, *(x[None, t: t + 1] for x in (q, k, v, g, beta)), state)[0])
    close(torch.cat(got), want, 2 * (T + D) * U, F32, "o")


def test_gdr_state_gates_at_their_ends_and_nan():
    """g = -inf forgets the state, beta = 0 writes nothing, and a NaN stays in its own sequence."""
    lens, H, D = [5, 6, 7], 2, 64
    q, k, v, g, beta, state, slots = gds_inputs(lens, H, H, D, D, F32, F32, 3, seed=3)
    g[2] = -float("inf")
    beta[5:8] = 0
    v[12, 0, 3] = float("nan")
    plan = api.make_gdr_state_plan(3, 18, H, D, D, dtype=F32)
    before = state.clone()
    cu = torch.tensor([0, 5, 11, 18], dtype=torch.int32, device="cuda")
    o = api.gdr_prefill(plan, q, k, v, g, beta, state, cu, slots=slots.cuda())
    tol = (7 + D) * U
    gds_check(lens[:2], q, k, v, g, beta, before, torch.where(torch.arange(3, device="cuda")[:, None, None, None] == int(slots[2]), before, state),
              o, slots[:2], None, D ** -0.5, tol, tol)
    bad = torch.isnan(state[int(slots[2])])
    assert bad[0, :, 3].all() and int(bad.sum()) == D  # the columns of the values are independent
    assert torch.isnan(o[12:, 0, 3]).all() and int(torch.isnan(o).sum()) == 6


@pytest.mark.parametrize("lens,sdt", [([4, 3, 2], BF16), ([6, 9, 5], BF16), ([4, 3, 2], F32)])
def test_gdr_few_tokens_keep_nan_and_resets_apart(lens, sdt):
    """In tiles of four tokens: what comes later, another sequence and another column do not reach a token."""
    H, D = 2, 128
    q, k, v, g, beta, state, slots = gds_inputs(lens, H, H, D, D, BF16, sdt, 3, seed=8)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    ends = [sum(lens[: i + 1]) - 1 for i in range(3)]
    g[1] = -float("inf")
    k[ends[0], 0, 5] = float("nan")     # the last key: its own output and the state
    v[ends[1], 1, 7] = float("inf")     # one column
    plan = api.make_gdr_state_plan(3, sum(lens), H, D, D, state_dtype=sdt)
    before = state.clone()
    o = api.gdr_prefill(plan, q, k, v, g, beta, state, cu, slots=slots.cuda())
    assert torch.isnan(o[ends[0], 0]).all() and torch.isnan(state[int(slots[0]), 0]).all()
    assert int((~torch.isfinite(o)).sum()) == D + 1
    q2, k2, v2 = (x.clone() for x in (q, k, v))
    k2[ends[0], 0, 5] = 0
    v2[ends[1], 1, 7] = 0
    again = before.clone()
    o2 = api.gdr_prefill(plan, q2, k2, v2, g, beta, again, cu, slots=slots.cuda())
    same = torch.isfinite(o)
    assert torch.equal(o[same], o2[same])
    gds_check(lens, q2, k2, v2, g, beta, before, again, o2, slots, None, D ** -0.5, (max(lens) + D) * U, (max(lens) + D) * U)


def test_gdr_state_refuses():
    plan = api.make_gdr_state_plan(2, 4, 2, 64, 64, dtype=F32)
    st = api.make_gdr_state(plan)
    q, k, v, g, beta, _, _ = gds_inputs([2, 2], 2, 2, 64, 64, F32, F32, 2)
    a = [x.unflatten(0, (2, 2)) for x in (q, k, v, g, beta)]
    for bad in (dict(slots=torch.zeros(3, device="cuda", dtype=torch.int32)), dict(slots=torch.zeros(2, device="cuda", dtype=torch.int64)),
                dict(fresh=torch.zeros(2, device="cuda")), dict(o=torch.empty(2, 2, 2, 32, device="cuda"))):
        with pytest.raises(ValueError):
            api.gdr_decode(plan, *a, st, **bad)
    with pytest.raises(ValueError):
        api.gdr_decode(plan, *a, st.to(BF16))
    with pytest.raises(ValueError):
        api.gdr_decode(plan, a[0].to(BF16), *a[1:], st)
    with pytest.raises(ValueError):
        api.gdr_decode(plan, *(x.expand(2, 4, *x.shape[2:]) if x.shape[1] == 1 else x.repeat(1, 2, *[1] * (x.dim() - 2)) for x in a), st)
    with pytest.raises(ValueError):
        api.gdr_prefill(plan, q, k, v, g, beta, st, torch.tensor([0, 4], device="cuda"))
    with pytest.raises(C.RmCpError) as e:
        api.make_gdr_state_plan(2, 4, 2, 48, 64)
    assert e.value.status == 4


# ------------------------------------------------------------------ norm of many tensors

def clip_ref(grads, max_norm, eps=1e-6):
    n = math.sqrt(sum(float(g.double().pow(2).sum()) for g in grads))
    return n, (min(1.0, max_norm / (n + eps)) if not math.isnan(n) else float("nan"))


def clip_case(sizes, types, seed=0, skew=1, std=1e-2):
    """Tensors that begin at odd addresses: views into one buffer a type."""
    out = []
    for i, n in enumerate(sizes):
        t = types[i % len(types)]
        out.append((std * rnd(n + 9, seed=seed + i)).to(t)[i * skew % 8: i * skew % 8 + n])
    return out


@pytest.mark.parametrize("sizes", [[1], [0, 3, 0], [16384, 16385, 16383, 1], [7, 100_003, 40_000, 0, 5, 77, 1_000_001], list(range(1, 200)),
                                   [3] * 2000], ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("types", [(F32,), (BF16,), (F32, BF16)], ids=["f32", "bf16", "mix"])
def test_clip_against_64_bits(sizes, types):
    grads = clip_case(sizes, types)
    want, coef = clip_ref(grads, 1e-3)
    plan = api.make_clip_plan(len(grads))
    # a square and the sum of at most 130 of them in fp32 (errors of both signs), fp64 beyond, one rounding
    assert abs(float(api.clip_grad_norm(plan, grads)) - want) <= 40 * U * want
    out = [torch.full_like(g, 7.0) for g in grads]
    norm = api.clip_grad_norm(plan, grads, 1e-3, out=out)
    assert abs(float(norm) - want) <= 40 * U * want
    cast = [torch.empty(g.numel(), device="cuda", dtype=BF16 if g.dtype == F32 else F32) for g in grads]
    api.clip_grad_norm(plan, grads, 1e-3, out=cast)
    inplace = [g.clone() for g in grads]
    api.clip_grad_norm(plan, inplace, 1e-3)
    for g, a, b, c in zip(grads, out, cast, inplace):
        if g.numel():
            w = g.double() * coef
            close(a, w, 44 * U, a.dtype, "out")
            close(b, w, 44 * U, b.dtype, "cast")
            assert torch.equal(a, c)


def test_clip_leaves_what_is_below_and_repeats_itself():
    grads = clip_case([50_000, 3, 999, 123_457], (F32, BF16))
    plan = api.make_clip_plan(8)
    before = [g.clone() for g in grads]
    n1 = api.clip_grad_norm(plan, grads, 1e6)
    for g, b in zip(grads, before):
        assert torch.equal(g, b)
    n2 = api.clip_grad_norm(plan, grads)
    assert torch.equal(n1, n2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n3 = api.clip_grad_norm(plan, grads, stream=side)
    side.synchronize()
    assert torch.equal(n1, n3)


@pytest.mark.parametrize("std", [1e30, 1e-30, 1e-42, 3e38])
def test_clip_norm_where_squares_leave_fp32(std):
    g = (rnd(30_001).clamp(-1, 1) * std).contiguous()
    want, _ = clip_ref([g], 1.0)
    got = float(api.clip_grad_norm(api.make_clip_plan(1), [g]))
    if want > 3.4e38:
        assert math.isinf(got)
    else:
        assert abs(got - want) <= 40 * U * want + 2.0 ** -149


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_clip_follows_the_formula_for_infinities_and_nan(bad):
    g = [rnd(1000), rnd(70_000, seed=1, dtype=BF16)]
    g[1][69_999] = bad
    out = [torch.empty_like(x) for x in g]
    norm = float(api.clip_grad_norm(api.make_clip_plan(2), g, 1.0, out=out))
    assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
    if math.isnan(bad):
        assert all(torch.isnan(x).all() for x in out)
    else:
        assert not out[0].any() and torch.isnan(out[1][-1]) and not out[1][:-1].any()


def test_clip_of_zeros_and_refusals():
    plan = api.make_clip_plan(2)
    z = torch.zeros(5000, device="cuda")
    assert float(api.clip_grad_norm(plan, [z], 1.0)) == 0.0 and not z.any()
    for bad in ([], [z, z, z], [z.half()], [z.view(50, 100).t()], [z.cpu()]):
        with pytest.raises(ValueError):
            api.clip_grad_norm(plan, bad, 1.0)
    with pytest.raises(ValueError):
        api.clip_grad_norm(plan, [z], 1.0, out=[z[:4]])
    with pytest.raises(ValueError):
        api.clip_grad_norm(plan, [z], out=[z])
    with pytest.raises(C.RmCpError):
        api.clip_grad_norm(plan, [z], -1.0)


def test_a_decoding_step_as_a_cuda_graph():
    """Norm with rotation, decoding and a norm of gradients captured once and replayed: the direct calls' values."""
    S, H, D = 3, 4, 128
    q, k, v, g, beta, state, slots = gds_inputs([1] * S, H, H, D, D, BF16, F32, S, seed=6)
    q, k, v, g, beta = (x.unflatten(0, (S, 1)) for x in (q, k, v, g, beta))
    table, pos, slots = api.make_rope_table(64, D), torch.tensor([[3], [9], [40]], dtype=torch.int32, device="cuda"), slots.cuda()
    plan, clip = api.make_gdr_state_plan(S, S, H, D, D), api.make_clip_plan(2)
    grads = [rnd(1000, seed=1), rnd(77, seed=2, dtype=BF16)]

    def step(st):
        a, b = api.qk_norm_rope(q, k, table, pos, norm="l2")
        return api.gdr_decode(plan, a, b, v, g, beta, st, slots=slots), api.clip_grad_norm(clip, grads)

    want_state = state.clone()
    want = [step(want_state) for _ in range(2)]
    held = state.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, norm = step(held)
    held.copy_(state)
    for w, wn in want:
        graph.replay()
        assert torch.equal(o, w) and torch.equal(norm, wn)
    assert torch.equal(held, want_state)
