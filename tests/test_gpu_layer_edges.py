"""Norm with rotation, the gated delta rule with a carried state, and clipping at the ends of what their
calls accept, against plain implementations in 64 bits (tolerances as in test_gpu_layer_ops.py)."""
import pytest
import torch

from state_summary_scan_gb300 import _capi as C
from state_summary_scan_gb300 import api
from test_gpu_layer_ops import BF16, F32, U, close, gds_check, gds_inputs, gds_ref, qkr_ref, rel2, rnd

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ norm and rotation

def qkr_case(B, T, Hq, Hk, D, R, dtype, fused=False, pos=None, weights=True, seed=0):
    if fused:
        x = (2 * rnd(B, T, (Hq + 2 * Hk) * D, seed=seed)).to(dtype)
        q, k = x[..., : Hq * D].unflatten(-1, (Hq, D)), x[..., Hq * D: (Hq + Hk) * D].unflatten(-1, (Hk, D))
    else:
        q, k = rnd(B, T, Hq, D, seed=seed, dtype=dtype), rnd(B, T, Hk, D, seed=seed + 1, dtype=dtype)
    table = api.make_rope_table(max(2000, T), R) if R else None
    p = None
    if pos:
        p = torch.randint(0, 2000, (B, T), generator=torch.Generator("cuda").manual_seed(seed + 2), device="cuda", dtype=pos)
    w = (1 + 0.3 * rnd(D, seed=seed + 3), 1 + 0.3 * rnd(D, seed=seed + 4)) if weights else (None, None)
    full = (torch.arange(T, device="cuda") if p is None else p.long()).expand(B, T)
    return q, k, dict(table=table, positions=p, q_weight=w[0], k_weight=w[1]), full


def pollute(n=64, floats=1 << 20):
    """Takes what the current stream's pool has free and writes NaN to it."""
    return [torch.full((floats >> (i % 12),), float("nan"), device="cuda") for i in range(n)]


@pytest.mark.parametrize("given", ["stream", "handle"])
def test_calls_on_another_stream_keep_their_buffers_to_themselves(given):
    """A call on a stream that is still busy: what the current stream allocates and writes after the call's
    return meets neither its workspace nor its outputs."""
    q, k, how, _ = qkr_case(1, 300, 4, 2, 128, 64, F32)
    dy = rnd(*q.shape, seed=7), rnd(*k.shape, seed=8)
    sq, sk, sv, g, beta, state, slots = gds_inputs([40], 2, 2, 64, 64, BF16, F32, 1)
    plan, clip = api.make_gdr_state_plan(1, 40, 2, 64, 64), api.make_clip_plan(1)
    cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")

    def calls(st, stream=None):
        a = api.qk_norm_rope(q, k, **how, stream=stream)
        b = api.qk_norm_rope_backward(q, k, *dy, **how, stream=stream)
        return *a, *b, api.gdr_prefill(plan, sq, sk, sv, g, beta, st, cu, stream=stream), api.clip_grad_norm(clip, [q], stream=stream)

    want = [x.clone() for x in calls(state.clone())]
    side = torch.cuda.Stream()
    for _ in range(3):
        st, junk = state.clone(), pollute()
        del junk  # free blocks of every size in the current stream's pool
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # some 10 ms
        got = calls(st, side if given == "stream" else side.cuda_stream)
        junk = pollute()
        side.synchronize()
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(got, want)):
            assert torch.equal(x, y), i


@pytest.mark.parametrize("handle", [0, 1])
def test_calls_take_the_default_streams_handles(handle):
    q, k, how, _ = qkr_case(1, 30, 4, 2, 128, 64, F32)
    want = api.qk_norm_rope(q, k, **how)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = api.qk_norm_rope(q, k, **how, stream=handle)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def qkr_check(q, k, how, pos, tol=32 * U, seed=9):
    """Forward and backward against 64 bits, with the tolerances of test_qkr_against_64_bits."""
    dtype, t64 = q.dtype, None if how["table"] is None else how["table"].double()
    got = api.qk_norm_rope(q, k, **how)
    dy = [rnd(*x.shape, seed=seed + i, dtype=dtype) for i, x in enumerate((q, k))]
    back = api.qk_norm_rope_backward(q, k, *dy, **how)
    for i, (x, w) in enumerate(((q, how["q_weight"]), (k, how["k_weight"]))):
        x64 = x.double().requires_grad_(True)
        w64 = None if w is None else w.double().requires_grad_(True)
        y = qkr_ref(x64, w64, t64, pos, how["norm"], how["eps"], how.get("interleaved", False))
        close(got[i], y.detach(), tol, dtype, f"output {i}")
        want = torch.autograd.grad(y, [x64] + ([] if w is None else [w64]), dy[i].double())
        close(back[i], want[0], 2 * tol, dtype, f"gradient {i}")
        if w is not None:
            n = x.numel() // x.shape[-1]
            scale = float((dy[i].double().abs() * 4).sum((0, 1, 2)).max())
            assert float((back[2 + i].double() - want[1]).abs().max()) <= (tol + n / 64 * U) * scale, f"weight {i}"


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("B,T,Hq,Hk,D,dtype", [(1, 5, 3, 1, 128, F32), (1, 5, 2, 2, 64, BF16), (2, 3, 1, 1, 80, F32), (1, 4001, 5, 5, 128, BF16),
                                               (1, 3700, 8, 9, 64, F32)], ids=str)
def test_qkr_without_eps(norm, B, T, Hq, Hk, D, dtype):
    """eps = 0: the rows that a group or a step of rows lacks have no say in the weights' gradients."""
    q, k, how, pos = qkr_case(B, T, Hq, Hk, D, D // 2, dtype)
    qkr_check(q, k, {**how, "norm": norm, "eps": 0.0}, pos)


@pytest.mark.parametrize("T", [3, 4000])
@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_qkr_gradient_of_tiny_rows(norm, T):
    """Rows of 3e-21 without eps: r is some 1e19 to 1e20, its square beyond fp32.  A square of 9e-42 is off by half of
    fp32's smallest number, 8e-5 of itself, r by half of that, and the gradient by three times r's error."""
    q, k, how, pos = qkr_case(1, T, 8, 8, 64, 32, F32)
    qkr_check(q * 3e-21, k * 3e-21, {**how, "norm": norm, "eps": 0.0}, pos, tol=3e-4)


@pytest.mark.parametrize("Hq,Hk,D", [(0, 2, 64), (2, 0, 64), (0, 0, 64), (2, 2, 0)])
def test_qkr_refuses_no_heads(Hq, Hk, D):
    """No heads of q and some of k: k' was never written."""
    q, k = rnd(1, 3, Hq, D), rnd(1, 3, Hk, D)
    with pytest.raises(ValueError):
        api.qk_norm_rope(q, k)
    with pytest.raises(ValueError):
        api.qk_norm_rope_backward(q, k, q, k)


LONG = [  # B, T, Hq, Hk, D, R, norm, weights, interleaved, dtype, fused, positions
    # enough tokens and heads for rows streamed through shared memory
    (1, 7297, 16, 16, 128, 128, "rms", True, False, BF16, False, None),
    (1, 8009, 8, 4, 128, 64, "l2", True, True, BF16, True, torch.int64),
    (3, 2501, 8, 9, 64, 64, "rms", True, False, F32, True, torch.int32),
    (2, 4001, 9, 5, 80, 48, "rms", True, False, F32, False, torch.int32),
    (1, 9001, 8, 8, 96, 96, "l2", False, True, BF16, False, None),
    (1, 7411, 16, 17, 32, 0, "rms", True, False, F32, False, None),
    (1, 16001, 4, 7, 256, 128, "none", True, False, BF16, True, torch.int32),
    (1, 7500, 4, 3, 256, 256, "rms", True, True, F32, False, torch.int64),
    # few heads, or pairs that straddle lanes: a loop over groups of heads, past a warp's first tokens
    (1, 20011, 2, 1, 64, 64, "rms", True, False, BF16, True, None),
    (1, 10001, 3, 2, 128, 128, "l2", True, True, F32, False, torch.int32),
    (1, 5003, 16, 2, 80, 20, "rms", True, False, BF16, False, torch.int32),
    (1, 2003, 5, 3, 128, 128, "rms", True, False, F32, True, torch.int32),
]


@pytest.mark.parametrize("case", LONG, ids=str)
def test_qkr_long_inputs_against_64_bits(case):
    B, T, Hq, Hk, D, R, norm, weights, inter, dtype, fused, pos = case
    q, k, how, full = qkr_case(B, T, Hq, Hk, D, R, dtype, fused, pos, weights)
    qkr_check(q, k, {**how, "norm": norm, "eps": 1e-5, "interleaved": inter}, full)


def test_qkr_long_inputs_with_rows_of_zeros_and_bad_positions():
    T, H, D, R = 8009, 16, 64, 32
    q, k = rnd(1, T, H, D), rnd(1, T, H, D, seed=1)
    q[0, 1] = 0
    k[0, T - 2, 3] = 0
    q[0, 2, 0, 5] = float("nan")
    table = api.make_rope_table(10, R)
    pos = torch.randint(0, 10, (T,), generator=torch.Generator("cuda").manual_seed(2), device="cuda", dtype=torch.int32)
    bad = torch.tensor([4, 700, 3648, T - 1], device="cuda")
    pos[bad] = torch.tensor([10, -1, 1 << 30, -(1 << 31)], device="cuda", dtype=torch.int32)
    how = dict(table=table, positions=pos, norm="l2", eps=1e-6)
    y, z = api.qk_norm_rope(q, k, **how)
    assert torch.equal(y[0, 1], torch.zeros_like(y[0, 1]))
    assert torch.isnan(y[0, 2, 0]).all() and not torch.isnan(y[0, 2, 1:]).any()
    for x in (y, z):
        assert torch.isnan(x[0, bad, :, :R]).all() and not torch.isnan(x[0, bad, :, R:]).any()
    fine = torch.ones(T, dtype=torch.bool, device="cuda")
    fine[bad] = False
    want = qkr_ref(k.double(), None, table.double(), pos.clamp(0, 9).long()[None], "l2", 1e-6, False)
    close(z[0, fine], want[0, fine], 32 * U, F32, "k'")
    dq, dk, _, _ = api.qk_norm_rope_backward(q, k, torch.ones_like(q), torch.ones_like(k), **how)
    assert torch.isnan(dk[0, bad]).all() and torch.isfinite(dk[0, fine]).all()
    fine[2] = False
    assert torch.isfinite(dq[0, fine]).all()


def test_qkr_adapter_refuses_second_derivatives():
    """The backward's result has no graph: a second derivative through it would be taken for 0."""
    q = rnd(1, 3, 2, 64).requires_grad_(True)
    y, z = api.qk_norm_rope_train(q, rnd(1, 3, 1, 64, seed=1), norm="l2")
    dq, = torch.autograd.grad((y * y * y).sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        (dq.square().sum() + q.square().sum()).backward()


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


KINDS = {  # Dk, Dv, dtype, state dtype: which kernels a call with the bound below goes through
    "fp32": (32, 40, F32, F32),
    "few": (128, 136, BF16, BF16),       # tiles of a bf16 state, up to four tokens
    "some": (64, 72, BF16, F32),
    "chunks": (128, 136, BF16, F32),
    "segments": (64, 64, BF16, F32),
}


def prefill_check(kind, lens, bound, begin=0, rest=0, padding=None):
    """Prompts that begin at token `begin` and leave `rest` tokens over, against 64 bits; two heads of one key head."""
    Dk, Dv, dtype, sdt = KINDS[kind]
    S, N = len(lens), begin + sum(lens) + rest
    q, k, v, g, beta, state, slots = gds_inputs([begin] + lens + [rest], 2, 1, Dk, Dv, dtype, sdt, S + 3)
    slots = slots[:S]
    if padding is not None:
        slots[padding] = -1
    plan = api.make_gdr_state_plan(S, N, 2, Dk, Dv, num_slots=S + 3, qk_heads=1, max_len=bound, dtype=dtype, state_dtype=sdt)
    cu = torch.tensor([begin] + lens).cumsum(0).to(torch.int32).cuda()
    before, o = state.clone(), torch.full_like(v, float("nan"))
    n0 = C.rm_cp_launch_count()
    api.gdr_prefill(plan, q, k, v, g, beta, state, cu, slots=slots.cuda(), max_len=bound, o=o)
    assert C.rm_cp_launch_count() - n0 == {"chunks": 2, "segments": 4}.get(kind, 1)
    assert C.rm_cp_device_status(torch.zeros(4, dtype=torch.int32, device="cuda")) == 0
    assert not o[:begin].any() and not o[N - rest:].any()
    if kind in ("fp32", "some"):
        tol, at = (max(lens) + Dk) * U, slice(begin, N - rest)
        gds_check(lens, q[at], k[at], v[at], g[at], beta[at], before, state, o[at], slots, None, Dk ** -0.5, tol, tol)
        return
    at, idle = begin, set(range(S + 3))
    for i, n in enumerate(lens):
        s, j = slice(at, at + n), int(slots[i])
        at += n
        if j < 0:
            assert not o[s].any()
            continue
        idle.discard(j)
        want_o, want_S = gds_ref(q[s], k[s], v[s], g[s], beta[s], before[j], Dk ** -0.5)
        if n:  # as in chunks; and a bf16 state rounded at most twice on the way to o: sqrt(3) of a rounding (1.7e-3)
            assert rel2(o[s], want_o) <= 2.0 ** -8, (i, rel2(o[s], want_o))
        assert rel2(state[j], want_S) <= 2e-3 + (2.0 ** -8 if sdt == BF16 else 0), (i, rel2(state[j], want_S))
    for j in idle:
        assert torch.equal(state[j], before[j])


@pytest.mark.parametrize("kind,lens,bound", [("fp32", [30, 5], 10), ("fp32", [7, 0, 3], 1), ("few", [9, 2, 4], 4), ("few", [6, 1], 1), ("some", [5, 3], 1),
                                             ("some", [30, 41], 7), ("chunks", [200, 30, 129], 64), ("chunks", [300], 48),
                                             ("segments", [4400, 5, 100], 3000)], ids=str)
def test_gdr_prefill_takes_prompts_over_the_bound(kind, lens, bound):
    prefill_check(kind, lens, bound)


@pytest.mark.parametrize("kind,lens,bound", [("fp32", [9, 0, 3], 9), ("few", [4, 0, 2], 4), ("some", [11, 12, 0], 12), ("chunks", [70, 0, 129], 129),
                                             ("segments", [0, 3100, 5], 3100)], ids=str)
@pytest.mark.parametrize("begin,rest", [(0, 5), (3, 200), (70, 0)])
def test_gdr_prefill_writes_zeros_for_tokens_of_no_prompt(kind, lens, bound, begin, rest):
    prefill_check(kind, lens, bound, begin, rest)
    prefill_check(kind, lens, bound, begin, rest, padding=0)
    prefill_check(kind, lens, bound, begin, rest, padding=len(lens) - 1)


def test_gdr_prefill_of_no_prompts():
    plan = api.make_gdr_state_plan(2, 100, 2, 64, 64)
    q, k, v, g, beta, state, _ = gds_inputs([10], 2, 2, 64, 64, BF16, F32, 2)
    before, o = state.clone(), torch.full_like(v, 7.0)
    api.gdr_prefill(plan, q, k, v, g, beta, state, torch.zeros(1, dtype=torch.int32, device="cuda"), o=o)
    assert not o.any() and torch.equal(state, before)


@pytest.mark.parametrize("bound", [None, 1, 64])
@pytest.mark.parametrize("sdt", [F32, BF16])
def test_gdr_prefill_of_empty_prompts_alone(bound, sdt):
    plan = api.make_gdr_state_plan(3, 100, 2, 64, 64, state_dtype=sdt)
    state = rnd(3, 2, 64, 64, dtype=sdt)
    before = state.clone()
    qkv = [torch.empty(0, 2, 64, device="cuda", dtype=BF16)] * 3
    gates = [torch.empty(0, 2, device="cuda")] * 2
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    fresh = torch.tensor([0, 1], dtype=torch.uint8, device="cuda")
    o = api.gdr_prefill(plan, *qkv, *gates, state, cu, fresh=fresh, max_len=bound)
    assert o.shape == (0, 2, 64)
    assert torch.equal(state[0], before[0]) and not state[1].any() and torch.equal(state[2], before[2])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [1, 3])
def test_gdr_strides_of_one_token_or_one_head_do_not_matter(dtype, n):
    """One token of rows, or one head of tokens, whose strides are not multiples of 16 bytes: no step is taken."""
    H = 2 if n == 1 else 1  # one of the two dimensions has one element
    row = 3 * 64 + 8

    def parts(seed):
        if n == 1:
            x = rnd(1, 3 * row, seed=seed, dtype=dtype).as_strided((1, H, row), (3 * row + 1, row, 1))
        else:
            x = rnd(n, row, seed=seed, dtype=dtype).as_strided((n, 1, row), (row, row + 1, 1))
        q, k, v = x[..., :64], x[..., 64: 128], x[..., 128: 192]
        assert any(s * q.element_size() % 16 for s in q.stride()[:2])
        return q, (k * 0.125).as_strided(k.shape, (H * 64, 64, 1)), v

    q, k, v = parts(1)
    g, beta, state = -rnd(n, H, seed=2).abs(), torch.sigmoid(rnd(n, H, seed=3)), rnd(1, H, 64, 64, seed=4)
    plan = api.make_gdr_state_plan(1, n, H, 64, 64, dtype=dtype)
    before, tol = state.clone(), (n + 64) * U
    o = api.gdr_prefill(plan, q, k, v, g, beta, state, torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    gds_check([n], q, k, v, g, beta, before, state, o, [0], None, 0.125, tol, tol)
    again = before.clone()
    o2 = api.gdr_decode(plan, *(x[None] for x in (q, k, v, g, beta)), again)
    assert torch.equal(o2[0], o) and torch.equal(again, state)


@pytest.mark.parametrize("Dk,Dv,sdt", [(64, 72, F32), (128, 128, F32), (128, 136, BF16)])
def test_gdr_prefill_as_a_recurrence_by_choice(Dk, Dv, sdt):
    """bf16 prompts that would run in chunks, at fp32's precision; a prompt's bits do not depend on its batch."""
    lens, H = [200, 7, 0, 64], 2
    q, k, v, g, beta, state, slots = gds_inputs(lens, H, 1, Dk, Dv, BF16, sdt, 5)
    how = dict(num_slots=5, qk_heads=1, state_dtype=sdt)
    plan = api.make_gdr_state_plan(4, sum(lens), H, Dk, Dv, recurrent=True, **how)
    assert C.rm_gdr_state_path(plan.c) == 0 and C.rm_gdr_state_path(api.make_gdr_state_plan(4, sum(lens), H, Dk, Dv, **how).c) == 1
    before, tol = state.clone(), (max(lens) + Dk) * U
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    o = api.gdr_prefill(plan, q, k, v, g, beta, state, cu, slots=slots.cuda())
    gds_check(lens, q, k, v, g, beta, before, state, o, slots, None, Dk ** -0.5, tol, tol)
    one = before.clone()
    o2 = api.gdr_prefill(plan, *(x[200:207] for x in (q, k, v, g, beta)), one, torch.tensor([0, 7], dtype=torch.int32, device="cuda"),
                         slots=slots[1:2].cuda())
    assert torch.equal(o2, o[200:207]) and torch.equal(one[int(slots[1])], state[int(slots[1])])


def chunked_check(lens, q, k, v, g, beta, before, after, o, slots, which=None):
    """In chunks, with the tolerances of test_gdr_prefill_in_chunks_against_64_bits."""
    at, sdt = 0, after.dtype
    for i, n in enumerate(lens):
        s, j = slice(at, at + n), int(slots[i])
        at += n
        if not 0 <= j < before.shape[0]:
            assert not o[s].any()
        elif n == 0:
            assert torch.equal(after[j], before[j])
        elif which is None or i in which:
            want_o, want_S = gds_ref(q[s], k[s], v[s], g[s], beta[s], before[j], q.shape[-1] ** -0.5)
            assert rel2(o[s], want_o) <= 2.0 ** -8, (i, rel2(o[s], want_o))
            assert rel2(after[j], want_S) <= 2e-3 + (2.0 ** -8 if sdt == BF16 else 0), (i, rel2(after[j], want_S))


@pytest.mark.parametrize("S,n,Dk,Dv", [(3, 48, 64, 64), (5, 65, 128, 72), (2, 130, 64, 256)])
def test_gdr_decode_of_many_tokens_in_chunks(S, n, Dk, Dv):
    q, k, v, g, beta, state, slots = gds_inputs([n] * S, 4, 2, Dk, Dv, BF16, F32, S + 2)
    slots[1] = -1
    plan = api.make_gdr_state_plan(S, S * n, 4, Dk, Dv, num_slots=S + 2, qk_heads=2, max_len=n)
    assert C.rm_gdr_state_path(plan.c) == 1
    before = state.clone()
    o = api.gdr_decode(plan, *(x.unflatten(0, (S, n)) for x in (q, k, v, g, beta)), state, slots=slots.cuda())
    chunked_check([n] * S, q, k, v, g, beta, before, state, o.flatten(0, 1), slots)


@pytest.mark.parametrize("S,Dk,Dv", [(33, 64, 64), (70, 128, 128), (1100, 64, 40)])
def test_gdr_prefill_of_many_prompts_in_chunks(S, Dk, Dv):
    lens = torch.randint(0, 140 if S < 1000 else 70, (S,), generator=torch.Generator().manual_seed(S)).tolist()
    lens[S // 2], lens[S - 1] = 0, 128
    q, k, v, g, beta, state, slots = gds_inputs(lens, 2, 1, Dk, Dv, BF16, F32, S + 2)
    slots[5] = S + 9
    plan = api.make_gdr_state_plan(S, sum(lens), 2, Dk, Dv, num_slots=S + 2, qk_heads=1, max_len=max(lens))
    before = state.clone()
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    o = api.gdr_prefill(plan, q, k, v, g, beta, state, cu, slots=slots.cuda())
    chunked_check(lens, q, k, v, g, beta, before, state, o, slots, range(0, S, 1 + S // 40))


@pytest.mark.parametrize("sdt", [F32, BF16])
@pytest.mark.parametrize("bound,launches", [(4100, 4), (6600, 4), (4100, 2)])
def test_gdr_prefill_at_128_through_strong_decay(sdt, bound, launches):
    """Strong chunks among weak ones, next to one another, at both ends of a segment and in the last chunk; in
    segments, and whole where the heads are many."""
    lens, H = [4100, 2500], 2 if launches == 4 else 40
    q, k, v, g, beta, state, slots = gds_inputs(lens, H, 1, 128, 128, BF16, sdt, 2, seed=4)
    g[300:420, 0] = -3.0
    g[900] = -float("inf")
    g[2000:2300, 1] *= 40
    g[4090:4100, 1] = -9.0   # the last tokens of the first prompt
    g[4500:4570, 0] = -4.0
    g[5000:5700:128, 1] = -70.0
    g[6000:6200, 1] = -0.95  # near the limit of a weak chunk
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    plan = api.make_gdr_state_plan(2, sum(lens), H, 128, 128, num_slots=2, qk_heads=1, state_dtype=sdt)
    before, n0 = state.clone(), C.rm_cp_launch_count()
    o = api.gdr_prefill(plan, q, k, v, g, beta, state, cu, slots=slots.cuda(), max_len=bound)
    assert C.rm_cp_launch_count() - n0 == launches
    chunked_check(lens, q, k, v, g, beta, before, state, o, slots)


# ------------------------------------------------------------------ what a call writes in place

def test_calls_raise_the_versions_of_what_they_write():
    """As in-place operations do, so that autograd sees that a saved tensor has changed."""
    plan, clip = api.make_gdr_state_plan(1, 10, 2, 64, 64), api.make_clip_plan(2)
    q, k, v, g, beta, state, _ = gds_inputs([10], 2, 2, 64, 64, BF16, F32, 1)
    a = [x[None] for x in (q, k, v, g, beta)]
    o, out, grads, clipped = torch.empty_like(a[2]), (torch.empty_like(a[0]), torch.empty_like(a[1])), [rnd(10), rnd(7)], [rnd(10), rnd(7)]
    with torch.inference_mode():
        kept = state.clone()  # has no version

    def changed(call, *tensors):
        before = [t._version for t in tensors]
        call()
        return [t._version > n for t, n in zip(tensors, before)]

    assert changed(lambda: api.gdr_decode(plan, *a, state, o=o), state, o, *a) == [True] * 2 + [False] * 5
    assert changed(lambda: api.gdr_decode(plan, *a, state), state, o) == [True, False]
    api.gdr_decode(plan, *a, kept)
    assert changed(lambda: api.qk_norm_rope(a[0], a[1], out=out), *out, *a) == [True] * 2 + [False] * 5
    assert changed(lambda: api.clip_grad_norm(clip, grads), *grads) == [False] * 2
    assert changed(lambda: api.clip_grad_norm(clip, grads, 1.0), *grads) == [True] * 2
    assert changed(lambda: api.clip_grad_norm(clip, grads, 1.0, out=clipped), *grads, *clipped) == [False] * 2 + [True] * 2
    w = rnd(10).requires_grad_(True)
    y = w * grads[0]
    api.clip_grad_norm(clip, grads, 1.0)
    with pytest.raises(RuntimeError):
        y.sum().backward()


# ------------------------------------------------------------------ offsets beyond 32 bits

@pytest.mark.parametrize("lens,dtype,sdt", [([1, 1], F32, F32), ([3, 2], F32, BF16), ([4, 1], BF16, BF16), ([9, 2], BF16, BF16), ([1, 1], BF16, F32),
                                            ([70, 5], BF16, F32), ([3100, 40], BF16, BF16)], ids=str)
def test_gdr_states_beyond_32_bits(lens, dtype, sdt):
    """The last slots of a pool of more than 2^31 elements; the first ones, where a 32-bit offset would lead, stay."""
    H, D = 2, 128
    slots_n = 2 ** 31 // (H * D * D) + 10
    q, k, v, g, beta, few, _ = gds_inputs(lens, H, 1, D, D, dtype, sdt, 20)
    state = torch.empty(slots_n, H, D, D, device="cuda", dtype=sdt)
    state[:10], state[-10:] = few[:10], few[10:]
    slots = torch.tensor([slots_n - 1, slots_n - 7], dtype=torch.int32)
    plan = api.make_gdr_state_plan(2, sum(lens), H, D, D, num_slots=slots_n, qk_heads=1, max_len=max(lens), dtype=dtype, state_dtype=sdt)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    o = api.gdr_prefill(plan, q, k, v, g, beta, state, cu, slots=slots.cuda())
    after, at = torch.cat([state[:10], state[-10:]]), torch.tensor([19, 13])
    if max(lens) >= 48:
        chunked_check(lens, q, k, v, g, beta, few, after, o, at)
        after[at] = few[at]
        assert torch.equal(after, few)
    else:
        tol = (max(lens) + D) * U
        gds_check(lens, q, k, v, g, beta, few, after, o, at, None, D ** -0.5, tol, tol)


@pytest.mark.parametrize("n,dtype,sdt", [(3, F32, F32), (3, BF16, BF16), (9, BF16, F32), (60, BF16, F32)], ids=str)
def test_gdr_tokens_beyond_32_bits(n, dtype, sdt):
    """Tokens that lie more than 2^31 elements apart."""
    H, D, step = 2, 64, (2 ** 31 // (n - 1) + 4096) // 8 * 8
    big = torch.empty((n - 1) * step + 8 * D, device="cuda", dtype=dtype)
    dense = gds_inputs([n], H, H, D, D, dtype, sdt, 1)
    q, k, v = (big.as_strided((n, H, D), (step, D, 1), 2 * i * D) for i in range(3))
    for to, x in zip((q, k, v), dense[:3]):
        to.copy_(x)
    g, beta, state = dense[3:6]
    plan = api.make_gdr_state_plan(1, n, H, D, D, dtype=dtype, state_dtype=sdt)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    one, two = state.clone(), state.clone()
    want = api.gdr_prefill(plan, *dense[:5], one, cu)
    assert torch.equal(api.gdr_prefill(plan, q, k, v, g, beta, two, cu), want) and torch.equal(one, two)


def test_gdr_outputs_beyond_32_bits():
    """65535 sequences of 132 heads of 256 values: only the last two have a state."""
    S, H, Dk, Dv = 65535, 132, 16, 256
    v = torch.empty(S, 1, H, Dv, device="cuda", dtype=BF16)
    assert v.numel() > 2 ** 31
    q, k, last, g, beta, state, _ = gds_inputs([1] * 2, H, 1, Dk, Dv, BF16, F32, 2)
    v[-2:, 0] = last
    slots = torch.full((S,), -1, dtype=torch.int32, device="cuda")
    slots[-2:] = torch.tensor([1, 0], dtype=torch.int32, device="cuda")

    def spread(x):
        y = torch.zeros(S, 1, *x.shape[1:], device="cuda", dtype=x.dtype)
        y[-2:, 0] = x
        return y

    plan = api.make_gdr_state_plan(S, S, H, Dk, Dv, num_slots=2, qk_heads=1, max_len=1)
    before = state.clone()
    o = api.gdr_decode(plan, spread(q), spread(k), v, spread(g), spread(beta), state, slots=slots)
    tol = (1 + Dk) * U
    gds_check([1, 1], q, k, last, g, beta, before, state, o[-2:, 0], [1, 0], None, Dk ** -0.5, tol, tol)
    assert not o[:-2].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_qkr_strides_beyond_32_bits(dtype):
    step = 2 ** 30 + 64
    big = torch.empty(2 * step + 512, device="cuda", dtype=dtype)
    q, k, how, pos = qkr_case(1, 3, 4, 2, 64, 32, dtype)
    far_q, far_k = big.as_strided(q.shape, (0, step, 64, 1)), big.as_strided(k.shape, (0, step, 64, 1), 256)
    far_q.copy_(q)
    far_k.copy_(k)
    dy = rnd(*q.shape, seed=7, dtype=dtype), rnd(*k.shape, seed=8, dtype=dtype)
    for a, b in zip(api.qk_norm_rope(far_q, far_k, **how), api.qk_norm_rope(q, k, **how)):
        assert torch.equal(a, b)
    for a, b in zip(api.qk_norm_rope_backward(far_q, far_k, *dy, **how), api.qk_norm_rope_backward(q, k, *dy, **how)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("R", [64, 20])
def test_qkr_rows_beyond_32_bits(R):
    """More than 2^31 elements of queries, through both forms for long inputs: the last tokens are as they are alone."""
    T, Hq, Hk, D = 2 ** 31 // (32 * 64) + 13, 32, 8, 64
    q = torch.randn(1, T, Hq, D, device="cuda", dtype=BF16, generator=torch.Generator("cuda").manual_seed(1))
    k = rnd(1, T, Hk, D, dtype=BF16)
    pos = torch.randint(0, 99, (1, T), device="cuda", dtype=torch.int32)
    table = api.make_rope_table(99, R)
    y, z = api.qk_norm_rope(q, k, table, pos)
    dq, dk, _, _ = api.qk_norm_rope_backward(q, k, y, z, table, pos)
    for at in (slice(0, 9), slice(T - 9, T)):
        cut = [x[:, at].contiguous() for x in (q, k, y, z, pos)]
        a, b = api.qk_norm_rope(cut[0], cut[1], table, cut[4])
        assert torch.equal(a, cut[2]) and torch.equal(b, cut[3])
        a, b, _, _ = api.qk_norm_rope_backward(*cut[:4], table, cut[4])
        close(dq[:, at], a, 64 * U, BF16, "dq")
        close(dk[:, at], b, 64 * U, BF16, "dk")


def test_clip_of_a_tensor_beyond_32_bits():
    n = 2 ** 31 + 1001
    g = torch.full((n,), 2.0 ** -10, device="cuda", dtype=BF16)
    g[-1000:] = 2.0 ** -3
    want = ((n - 1000) * 2.0 ** -20 + 1000 * 2.0 ** -6) ** 0.5
    norm = float(api.clip_grad_norm(api.make_clip_plan(1), [g], want / 2))
    assert abs(norm - want) <= 40 * U * want
    # the factor is a half but for eps: half of a power of two, rounded to bf16
    assert bool((g[-1000:] == 2.0 ** -4).all()) and bool((g[:-1000] == 2.0 ** -11).all())
