"""Linear attention on a pool of states at the ends of what the calls accept."""
import math

import pytest
import torch
from test_gpu_gla_state import BF, F32, check, make, plan_of, prefill, reference

from state_summary_scan_gb300 import RmCpError, api
from state_summary_scan_gb300 import _capi as C

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,Hqk,Dk,Dv", [(2, 1, 128, 128), (4, 4, 64, 72)])
def test_nothing_of_a_neighbour_is_used(H, Hqk, Dk, Dv, dtype):
    """Tokens of no sequence, padding sequences and other slots hold NaN: outputs there are 0, the slots stay as they are."""
    lens = [70, 3, 130, 0, 65]
    x, slots, fresh, cu = make(lens, H, Hqk, Dk, Dv, dtype, F32, extra=(67, 70))
    slots[2] = 99  # a padding sequence
    for n in ("q", "k", "v", "g"):
        x[n][:67] = float("nan")
        x[n][cu[2]: cu[3]] = float("nan")
        x[n][cu[-1]:] = float("nan")
    other = [i for i in range(x["state"].shape[0]) if i not in slots.tolist()]
    x["state"][other] = float("nan")
    want = reference({k: t.nan_to_num() for k, t in x.items()}, slots, fresh, cu, Dk)
    o, state, plan = prefill(x, slots, fresh, cu, lens, H, Hqk, Dk, Dv)
    assert bool((o[:67] == 0).all()) and bool((o[cu[-1]:] == 0).all()) and bool((o[cu[2]: cu[3]] == 0).all())
    assert bool(state[other].isnan().all())
    keep = [s for i, s in enumerate(slots.tolist()) if i != 2]
    check(o, state[keep], (want[0], want[1][keep], want[2], want[3][keep]), lens, Dk, dtype, F32, C.rm_cp_gla_state_path(plan.c) == 1)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_an_empty_prompt_leaves_its_slot_or_a_zero_state(dtype):
    x, slots, _, cu = make([0, 40, 0], 2, 2, 64, 64, dtype, BF)
    fresh = torch.tensor([1, 0, 0], dtype=torch.uint8)
    before = x["state"].clone()
    _, state, _ = prefill(x, slots, fresh, cu, [0, 40, 0], 2, 2, 64, 64)
    assert bool((state[slots[0]] == 0).all()) and torch.equal(state[slots[2]].cpu(), before[slots[2]])


@pytest.mark.parametrize("max_len", [1, 4, 40, 64, 1000])
@pytest.mark.parametrize("dtype,state_dtype", [(BF, F32), (F32, F32), (BF, BF)])
def test_a_prompt_longer_than_its_bound_is_taken_whole(max_len, dtype, state_dtype):
    lens = [1300, 5, 0, 66]
    x, slots, fresh, cu = make(lens, 1, 1, 128, 64, dtype, state_dtype, "head", seed=4)
    plan = api.make_gla_state_plan(4, 1371, 1, 128, 64, num_slots=6, dtype=dtype, state_dtype=state_dtype)
    d = {n: t.cuda() for n, t in x.items()}
    o = api.gla_prefill(plan, d["q"], d["k"], d["v"], d["g"], d["state"], cu.cuda(), slots=slots.cuda(), fresh=fresh.cuda(), max_len=max_len)
    chunks = dtype == BF and max_len >= 32
    want = reference(x, slots, fresh, cu, 128)
    if state_dtype == BF and max_len <= 4:  # rounded every four tokens: 2^-8 of the state each time, under decays that keep some 1 / 0.6 of them
        err = (d["state"].double().cpu() - want[1]).abs()
        assert bool((err <= 2.0 ** -8 * 3 * want[3] + 1e-30).all())
        return
    check(o, d["state"], want, lens, 128, dtype, state_dtype, chunks)


def test_slices_of_a_projection_and_odd_strides():
    """q, k and v read in place, g with a token stride of its own; the same results as of contiguous copies."""
    H, Dk, Dv, N = 4, 64, 64, 200
    g = torch.Generator().manual_seed(3)
    wide = torch.randn(N, 3 * H * 64 + 64, generator=g).to(BF).cuda()
    q, k, v = (wide[:, 32 + i * H * 64: 32 + (i + 1) * H * 64].unflatten(-1, (H, 64)) for i in range(3))
    gate = torch.nn.functional.logsigmoid(torch.randn(N, 3 * H, generator=g) + 3).cuda()[:, H: 2 * H]
    plan = api.make_gla_state_plan(2, N, H, Dk, Dv, max_len=130)
    cu = torch.tensor([0, 130, 200], dtype=torch.int32, device="cuda")
    a, b = api.make_gla_state(plan), api.make_gla_state(plan)
    o = api.gla_prefill(plan, q, k, v, gate, a, cu)
    p = api.gla_prefill(plan, q.contiguous(), k.contiguous(), v.contiguous(), gate.contiguous(), b, cu)
    assert torch.equal(o, p) and torch.equal(a, b)
    # head-major inputs
    o = api.gla_prefill(plan, *(t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)), gate, a.zero_(), cu)
    assert torch.equal(o, p) and torch.equal(a, b)
    # decoding: token by token from the same projection
    o = api.gla_decode(plan, q[:2, None], k[:2, None], v[:2, None], gate[:2, None], a, slots=None)
    p = api.gla_decode(plan, q[:2, None].contiguous(), k[:2, None].contiguous(), v[:2, None].contiguous(), gate[:2, None].contiguous(), b)
    assert torch.equal(o, p) and torch.equal(a, b)


@pytest.mark.parametrize("state_dtype", [F32, BF])
def test_prefill_then_decoding_continues_the_state(state_dtype):
    """A prompt in chunks, then tokens one, three and two at a time, against one recurrence over all of them."""
    H, Hqk, D, lens, more = 2, 1, 128, [150, 33], [1, 3, 2]
    x, slots, fresh, cu = make([n + sum(more) for n in lens], H, Hqk, D, D, BF, state_dtype, "token", seed=6)
    fresh[:] = 1
    plan = plan_of(x, [200, 200], H, Hqk, D, D)
    d = {n: t.cuda() for n, t in x.items()}
    rows = [torch.arange(cu[i], cu[i + 1]) for i in range(2)]
    first = torch.cat([r[:n] for r, n in zip(rows, lens)])
    pick = lambda at: [d[n][at.cuda()] for n in ("q", "k", "v", "g")]  # noqa: E731
    o = torch.zeros_like(d["v"])
    c = torch.tensor([0, *lens]).cumsum(0).int().cuda()
    o[first] = api.gla_prefill(plan, *pick(first), d["state"], c, slots=slots.cuda(), fresh=fresh.cuda(), max_len=150)
    at = 0
    for n in more:
        now = torch.stack([r[m + at: m + at + n] for r, m in zip(rows, lens)])
        o[now.flatten()] = api.gla_decode(plan, *pick(now), d["state"], slots=slots.cuda()).flatten(0, 1)
        at += n
    ro, rs, A, B = reference(x, slots, fresh, cu, D)
    # three hand-overs round a bf16 pool by 2^-8 of it each, which reaches the outputs too
    hand = 4 * 2.0 ** -8 if state_dtype == BF else 0.0
    err = (o.double().cpu() - ro).abs()
    assert bool((err <= (2.2 * 2.0 ** -8 + hand) * A + 2.0 ** -8 * ro.abs() + 1e-30).all())
    err = (d["state"].double().cpu() - rs).abs()
    assert bool((err <= (hand + 64 * 2.0 ** -24 * 4) * B + (2.0 ** -8 * rs.abs() if state_dtype == BF else 0) + 1e-30).all())


@pytest.mark.parametrize("n", [1, 70])
def test_strong_and_absent_decays(n):
    """g = 0 keeps everything, -inf nothing, positive gates grow; a NaN reaches its own sequence's later tokens alone."""
    H, D, S = 5, 64, 3
    x, slots, fresh, cu = make([n] * S, H, H, D, D, BF, F32, "token", seed=9)
    x["g"][:, 0], x["g"][:, 1], x["g"][:, 2], x["g"][:, 3] = 0.0, -math.inf, 0.05, -1e30
    x["g"][n, 4] = float("nan")  # the second sequence's first token
    o, state, _ = prefill(x, slots, fresh, cu, [n] * S, H, H, D, D)
    clean = {k: t.clone() for k, t in x.items()}
    clean["g"][n, 4] = 0
    ro, rs, A, B = reference(clean, slots, fresh, cu, D)
    assert bool(o[n: 2 * n, 4].isnan().all()) and bool(state[slots[1], 4].isnan().all())
    o[n: 2 * n, 4], state[slots[1], 4] = ro[n: 2 * n, 4].to(BF).cuda(), rs[slots[1], 4].float().cuda()
    check(o, state, (ro, rs, A, B), [n] * S, D, BF, F32, n >= 64)


def test_a_nan_in_a_token_stays_in_its_sequence():
    lens = [100, 90, 64]
    for name in ("q", "k", "v"):
        x, slots, fresh, cu = make(lens, 2, 2, 128, 128, BF, F32, seed=2)
        good, state, _ = prefill({k: t.clone() for k, t in x.items()}, slots, fresh, cu, lens, 2, 2, 128, 128)
        x[name][150] = float("nan")  # token 50 of the second prompt
        o, after, _ = prefill(x, slots, fresh, cu, lens, 2, 2, 128, 128)
        assert torch.equal(o[:100], good[:100]) and torch.equal(o[190:], good[190:])
        assert all(torch.equal(after[s], state[s]) for s in (slots[0], slots[2]))
        assert bool(o[150].isnan().any())


def test_graphs_streams_and_version_counters():
    lens = [90, 1000, 4]
    x, slots, fresh, cu = make(lens, 2, 2, 64, 128, BF, F32, seed=7)
    plan = plan_of(x, lens, 2, 2, 64, 128)
    d = {n: t.cuda() for n, t in x.items()}
    start = d["state"].clone()
    args = (d["q"], d["k"], d["v"], d["g"])
    kw = dict(slots=slots.cuda(), fresh=fresh.cuda())
    v = d["state"]._version
    want = api.gla_prefill(plan, *args, d["state"], cu.cuda(), **kw)
    assert d["state"]._version > v
    end, c = d["state"].clone(), cu.cuda()
    s = torch.cuda.Stream()
    d["state"].copy_(start)
    s.wait_stream(torch.cuda.current_stream())
    got = api.gla_prefill(plan, *args, d["state"], c, stream=s, **kw)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(d["state"], end)
    o = torch.empty_like(want)
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            api.gla_prefill(plan, *args, d["state"], c, o=o, **kw)
    for _ in range(2):
        d["state"].copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(d["state"], end)
    torch.cuda.synchronize()
    scratch = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert C.rm_cp_device_status(scratch) == 0  # no wait ran out


def test_calls_without_sequences_or_tokens():
    plan = api.make_gla_state_plan(3, 64, 2, 64, 64)
    state = api.make_gla_state(plan).fill_(1)
    q = torch.zeros(0, 2, 64, dtype=BF, device="cuda")
    g = torch.zeros(0, 2, device="cuda")
    o = api.gla_prefill(plan, q, q, q, g, state, torch.zeros(4, dtype=torch.int32, device="cuda"), fresh=torch.tensor([0, 1, 0], dtype=torch.uint8, device="cuda"))
    assert o.shape == (0, 2, 64) and bool((state[1] == 0).all()) and bool((state[0] == 1).all()) and bool((state[2] == 1).all())
    q = torch.ones(5, 2, 64, dtype=BF, device="cuda")
    o = api.gla_prefill(plan, q, q, q, torch.zeros(5, 2, device="cuda"), state, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert bool((o == 0).all())


def test_offsets_beyond_2_31_elements():
    """The pool's last slots and the last tokens of large inputs."""
    H, D, slots_n = 16, 128, 8400  # 2.2e9 elements of state
    plan = api.make_gla_state_plan(2, 256, H, D, D, num_slots=slots_n, state_dtype=BF)
    state = torch.zeros(slots_n, H, D, D, dtype=BF, device="cuda")
    gen = torch.Generator("cuda").manual_seed(1)
    q, k, v = (torch.randn(200, H, D, generator=gen, device="cuda").to(BF) for _ in range(3))
    g = torch.full((H,), -0.1, device="cuda")
    cu = torch.tensor([0, 130, 200], dtype=torch.int32, device="cuda")
    far = torch.tensor([slots_n - 1, slots_n - 3], dtype=torch.int32, device="cuda")
    o = api.gla_prefill(plan, q, k, v, g, state, cu, slots=far)
    small = torch.zeros(2, H, D, D, dtype=BF, device="cuda")
    near = api.make_gla_state_plan(2, 256, H, D, D, state_dtype=BF)
    p = api.gla_prefill(near, q, k, v, g, small, cu)
    assert torch.equal(o, p) and torch.equal(state[far.long()], small)
    assert bool((state[slots_n - 2] == 0).all()) and bool((state[0] == 0).all())
    one = lambda t: t[:2, None].contiguous()  # noqa: E731
    assert torch.equal(api.gla_decode(plan, one(q), one(k), one(v), g, state, slots=far), api.gla_decode(near, one(q), one(k), one(v), g, small))
    assert torch.equal(state[far.long()], small)


@pytest.mark.parametrize("bad", ["dtype", "state", "g", "g heads", "tokens", "slots", "cu", "Dk"])
def test_refusals(bad):
    if bad == "Dk":
        with pytest.raises(RmCpError):
            api.make_gla_state_plan(1, 8, 2, 48, 64, device="cuda")
        return
    plan = api.make_gla_state_plan(2, 64, 2, 64, 64)
    q = torch.zeros(64, 2, 64, dtype=BF, device="cuda")
    a = dict(q=q, k=q, v=q, g=torch.zeros(64, 2, device="cuda"), state=api.make_gla_state(plan), cu_seqlens=torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda"))
    kw = {}
    if bad == "dtype":
        a["q"] = q.float()
    elif bad == "state":
        a["state"] = a["state"].to(BF)
    elif bad == "g":
        a["g"] = a["g"].to(BF)
    elif bad == "g heads":
        a["g"] = torch.zeros(3, device="cuda")
    elif bad == "tokens":
        a["q"] = a["k"] = a["v"] = torch.zeros(65, 2, 64, dtype=BF, device="cuda")
        a["g"] = torch.zeros(65, 2, device="cuda")
    elif bad == "slots":
        kw["slots"] = torch.zeros(3, dtype=torch.int32, device="cuda")
    else:
        a["cu_seqlens"] = a["cu_seqlens"].long()
    with pytest.raises(ValueError):
        api.gla_prefill(plan, **a, **kw)




@pytest.mark.parametrize("state_dtype", [F32, BF])
@pytest.mark.parametrize("short", [(128, 129), (127, 320), (321, 64), (1, 512), (0, 1217)])
def test_prompts_that_end_where_segments_do(short, state_dtype):
    """1280 tokens are cut after 2 chunks, and then after every 3: tokens 128, 320, 512, ..., 1088."""
    lens = [short[0], 1280, short[1]]
    x, slots, fresh, cu = make(lens, 1, 1, 64, 128, BF, state_dtype, seed=sum(short))
    o, state, plan = prefill(x, slots, fresh, cu, lens, 1, 1, 64, 128)
    assert C.rm_cp_gla_state_path(plan.c) == 1
    check(o, state, reference(x, slots, fresh, cu, 64), lens, 64, BF, state_dtype, True)
