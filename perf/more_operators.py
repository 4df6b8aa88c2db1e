"""Cases that measure linear attention served from a pool of states, and the norms around a mixer:

  gla   linear attention with a decay for each head and a carried state: recurrent (a few tokens for
        each of many sequences, state updated in place) and ragged prefill (whole prompts)
  rms   root-mean-square norm with the residual's addition: with an output in 8 bits and scales
        (serving), or in the input's type with its backward (training); with a gate, the norm of a
        mixer's outputs

run() computes an operator in its plain form (elementary torch operations in 32 bits) or, where
`own` is set, through the framework's entry points.  exact() computes the same from the
definition in 64 bits.
"""
import math
import random

import torch

own = False

F = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
F8_MAX = 448.0  # the largest e4m3 value
TINY = 2.0 ** -126  # the smallest scale


# ------------------------------------------------------------------------------ the cases

def _gla(name, S, n, H, Hqk, Dk, Dv, **kw):
    # n: tokens of each sequence (decode) or the longest sequence (prefill); gate: a decay for each token of
    # a head, or one for the head
    c = dict(op="gla", mode="decode", S=S, n=n, H=H, Hqk=Hqk, Dk=Dk, Dv=Dv, dtype="bf16", state="f32", gate="token",
             lens=0, fresh=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def _rms(name, N, H, n, **kw):
    # N tokens of H rows of n elements; residual: its type, or none; group: elements of a scale (0: the row,
    # -1: no output in 8 bits)
    c = dict(op="rms", N=N, H=H, n=n, dtype="bf16", residual="none", gate=False, gate_first=False, weight=True, group=-1,
             backward=False, fused=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one sequence, one token, the 64-wide heads of the 8k configuration: the smallest call
        _gla("gla decode 1", 1, 1, 16, 16, 64, 64),
        # a batch of users, one token each, 128-wide heads, a fixed decay for each head
        _gla("gla decode 256", 256, 1, 16, 16, 128, 128, gate="head"),
        # several tokens checked at a time, bf16 state, heads sharing queries and keys, wide values
        _gla("gla decode 4 tokens", 61, 4, 32, 16, 128, 256, state="bf16"),
        # a fp32 model of odd sizes, ragged prompts with an empty and a one-token one
        _gla("gla prefill fp32", 7, 301, 6, 3, 32, 40, mode="prefill", dtype="f32", lens=3),
        # one 8k prompt of 128-wide heads, a fixed decay for each head
        _gla("gla prefill 8k", 1, 8192, 16, 16, 128, 128, mode="prefill", gate="head", fresh=True),
        # ragged prompts of a batch, heads sharing queries and keys, some continuing a state
        _gla("gla prefill ragged", 13, 4096, 32, 16, 128, 128, mode="prefill", state="bf16", lens=5, fresh=True),
        # a decoding step's block norm before a projection in 8 bits, a scale for each token: latency
        _rms("rms decode 8 bits", 32, 1, 2048, residual="bf16", group=0),
        # the same for a batch of prompts, a scale for each 128 elements
        _rms("rms prefill 8 bits", 8191, 1, 4096, residual="bf16", group=128),
        # the training step of the 32k configuration, 16 heads of 128: the norm before its projections
        _rms("rms train 32k", 32768, 1, 2048, residual="bf16", backward=True),
        # a fp32 training step of a small model of odd sizes
        _rms("rms train fp32", 2047, 1, 1000, dtype="f32", residual="f32", backward=True),
        # the gated norm of a mixer's outputs in decoding, before a projection in 8 bits
        _rms("gated rms decode 8 bits", 61, 16, 128, gate=True, group=128, fused=True),
        # the gated norm in the training step of the 32k configuration, the gate a slice of a projection
        _rms("gated rms train 32k", 32768, 16, 128, gate=True, backward=True, fused=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "rms", "rms", "gated"])
    gate = rng.choice(["token", "token", "head"])
    if op == "decode":
        Dk, Dv = rng.choice([(64, 64), (128, 128), (128, 256), (32, 48), (128, 64), (64, 128)])
        Hqk = rng.choice([2, 4, 8, 16])
        H = Hqk * rng.choice([1, 2])
        S = _log(rng, 1, max(1, min(512, (256 * 16 * 128 * 128) // (H * Dk * Dv))))
        return _gla(None, S, rng.choice([1, 1, 1, 2, 3, 5, 8]), H, Hqk, Dk, Dv, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    state="f32" if rng.random() < 0.6 else "bf16", gate=gate, fresh=rng.random() < 0.3)
    if op == "prefill":
        f32 = rng.random() < 0.3
        S = _log(rng, 1, 16)
        Hqk = rng.choice([2, 4, 8, 16])
        H = Hqk * rng.choice([1, 2]) if Hqk < 16 else 16
        Dk, Dv = rng.choice([(64, 64), (128, 128), (128, 256), (32, 48), (64, 128)])
        most = min(4096, (4096 * 13 * 32 * 128 * 128) // (S * H * Dk * Dv))
        return _gla(None, S, _log(rng, 2, 500 if f32 else most), H, Hqk, Dk, Dv, mode="prefill", dtype="f32" if f32 else "bf16",
                    state="f32" if f32 else rng.choice(["f32", "bf16"]), gate=gate, lens=rng.randrange(1, 1000), fresh=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    kind = rng.choice(["plain", "8 bits", "train"])
    if op == "rms":
        n = rng.choice([256, 512, 1000, 1024, 1536, 2048, 2560, 4096, 5120, 8192])
        residual = rng.choice(["none", dtype, dtype, "f32"])
        N = _log(rng, 1, min(32768, 32768 * 2048 // n) // (2 if "f32" in (dtype, residual) else 1))
        return _rms(None, N, 1, n, dtype=dtype, residual=residual, weight=rng.random() < 0.8,
                    group=rng.choice([0, 0, 128, 64, 32] if n % 128 == 0 else [0]) if kind == "8 bits" else -1, backward=kind == "train")
    n, H = rng.choice([64, 96, 128, 128, 256]), rng.choice([1, 2, 6, 8, 16])
    N = _log(rng, 1, 32768 * 16 * 128 // (n * H) // (4 if dtype == "f32" else 2))
    return _rms(None, N, H, n, dtype=dtype, gate=True, gate_first=rng.random() < 0.4, weight=rng.random() < 0.8,
                group=rng.choice([0, 32] + ([64, n] if n in (64, 128) else [])) if kind == "8 bits" else -1, backward=kind == "train",
                fused=rng.random() < 0.5)


def _lens(case):
    """Lengths of a prefill's sequences: from the case alone, an empty and a one-token one among many."""
    r = random.Random(case["lens"])
    lens = [r.randint(1, case["n"]) for _ in range(case["S"])]
    lens[r.randrange(case["S"])] = case["n"]
    if case["S"] > 4:
        at = [i for i in range(case["S"]) if lens[i] != case["n"]][:2]
        for i, n in zip(at, (0, 1)):
            lens[i] = n
    return lens


# ------------------------------------------------------------------------------ the inputs

def _prepare_gla(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    S, n, H, Hqk, Dk, Dv = (case[x] for x in ("S", "n", "H", "Hqk", "Dk", "Dv"))
    rnd = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    prefill = case["mode"] == "prefill"
    lens = _lens(case) if prefill else [n] * S
    N = sum(lens)
    dt, st = F[case["dtype"]], F[case["state"]]
    k = rnd(N, Hqk, Dk)
    k = (k / k.norm(dim=-1, keepdim=True)).to(dt)
    slots = S + 3  # the pool has room for others
    s = {"op": "gla", "case": case, "q": rnd(N, Hqk, Dk).to(dt), "k": k, "v": rnd(N, H, Dv).to(dt),
         "state": (0.3 * rnd(slots, H, Dk, Dv)).to(st),
         "slots": torch.randperm(slots, generator=gen, device=dev)[:S].to(torch.int32),
         "lens": lens, "scale": Dk ** -0.5, "fresh": None}
    if case["gate"] == "token":  # log-decays of a data-dependent gate
        s["g"] = torch.nn.functional.logsigmoid(rnd(N, H) + 4)
    else:  # one for each head, from a memory of two tokens to one of some thousand
        s["g"] = -torch.logspace(math.log10(0.5), -3, H, device=dev) * (1 + 0.1 * torch.rand(H, generator=gen, device=dev))
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    if case["fresh"]:  # every other sequence begins
        s["fresh"] = (torch.arange(S, device=dev) % 2 == 0).to(torch.uint8)
    if not prefill:
        for x in ("q", "k", "v") + (("g",) if case["gate"] == "token" else ()):
            s[x] = s[x].unflatten(0, (S, n))
    if own:
        from state_summary_scan_gb300 import api
        s["plan"] = api.make_gla_state_plan(S, N, H, Dk, Dv, num_slots=slots, qk_heads=Hqk, max_len=max(lens), scale=s["scale"],
                                            dtype=dt, state_dtype=st, device=dev)
    return s


def _prepare_rms(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    N, H, n, dt = case["N"], case["H"], case["n"], F[case["dtype"]]
    rnd = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    shape = (N, H, n) if case["gate"] else (N, n)
    s = {"op": "rms", "case": case, "x": rnd(*shape).to(dt), "residual": None, "z": None, "w": None}
    if case["residual"] != "none":  # a residual stream: a few of its elements are far larger than the others
        big = 1 + 30 * (torch.rand(n, generator=gen, device=dev) < 0.005)
        s["residual"] = (3 * rnd(*shape) * big).to(F[case["residual"]])
    if case["gate"]:
        if case["fused"]:  # the gate's part of one projection of queries, keys, values and gates
            s["z"] = rnd(N, 4 * H * n).to(dt)[:, 3 * H * n:].unflatten(-1, (H, n))
        else:
            s["z"] = rnd(N, H, n).to(dt)
    if case["weight"]:
        s["w"] = 1 + 0.2 * rnd(n)
    if case["backward"]:
        s["dy"] = rnd(*shape).to(dt)
        s["dh"] = rnd(*shape).to(s["residual"].dtype) if s["residual"] is not None else None
    return s


def prepare(case, seed):
    return {"gla": _prepare_gla, "rms": _prepare_rms}[case["op"]](case, seed)


# ------------------------------------------------------------------------------ the plain forms

def _plain_gla(s):
    """In chunks of up to 64 tokens: the scores within each, and the states before each from what the chunks write."""
    case = s["case"]
    S, H, Hqk, L = case["S"], case["H"], case["Hqk"], max(s["lens"])
    C = min(L, 64)
    n = -(-L // C)
    prefill = case["mode"] == "prefill"
    dev = s["q"].device
    at = torch.arange(n * C, device=dev)[None, :] + s["cu"][:-1, None]  # padded: a token past a sequence's end changes nothing
    live = at < s["cu"][1:, None]
    at = torch.where(live, at, 0).long()

    def chunks(x):  # [S, heads, chunks, C, ...]
        x = x if prefill else x.flatten(0, 1)
        x = torch.where(live.view(S, n * C, *[1] * (x.dim() - 1)), x[at], 0)
        return x.unflatten(1, (n, C)).movedim(3, 1)

    gate = s["g"] if case["gate"] == "token" else s["g"].expand(*s["q"].shape[:-2], H)
    q, k, v = (chunks(s[x]).float() for x in ("q", "k", "v"))
    q, k = q.repeat_interleave(H // Hqk, 1) * s["scale"], k.repeat_interleave(H // Hqk, 1)
    b = chunks(gate).double().cumsum(-1)  # from the chunk's start
    end = b[..., -1].cumsum(-1)  # [S, H, chunks]: from the sequence's
    begin = torch.cat([torch.zeros_like(end[..., :1]), end], -1)
    below = torch.ones(C, C, dtype=torch.bool, device=dev).tril()
    gap = torch.where(below, b[..., :, None] - b[..., None, :], -math.inf).exp().float()
    o = torch.matmul(torch.matmul(q, k.mT) * gap, v)
    wrote = torch.matmul((k * (b[..., -1:] - b).exp().float()[..., None]).mT, v)  # [S, H, chunks, Dk, Dv]
    before = torch.ones(n + 1, n, dtype=torch.bool, device=dev).tril(-1)
    fade = torch.where(before, begin[..., :, None] - end[..., None, :], -math.inf).exp().float()
    slots = s["slots"].long()
    first = s["state"][slots].float()
    if s["fresh"] is not None:
        first = torch.where(s["fresh"].view(S, 1, 1, 1) != 0, 0.0, first)
    states = torch.matmul(fade, wrote.flatten(-2)).unflatten(-1, first.shape[-2:]) + begin.exp().float()[..., None, None] * first[:, :, None]
    o = o + b.exp().float()[..., None] * torch.matmul(q, states[:, :, :-1])
    o = o.movedim(1, 3).flatten(1, 2)[:, :L].to(s["v"].dtype)
    s["state"][slots] = states[:, :, -1].to(s["state"].dtype)
    return {"o": o[live[:, :L]] if prefill else o, "state": s["state"]}


def _plain_rms(s):
    case, eps = s["case"], 1e-6
    x, z, w = s["x"].float(), s["z"], s["w"]
    res = {}
    h = x
    if s["residual"] is not None:
        res["h"] = (x + s["residual"].float()).to(s["residual"].dtype)
        h = res["h"].float()
    if z is not None:
        z = z.float()
        sig = 1 / (1 + (-z).exp())
        act = z * sig
    u = h * act if z is not None and case["gate_first"] else h
    r = torch.rsqrt((u * u).mean(-1, keepdim=True) + eps)
    m = u * r if w is None else u * r * w
    y = m * act if z is not None and not case["gate_first"] else m
    if case["group"] < 0:
        res["y"] = y.to(s["x"].dtype)
    else:
        y = y.unflatten(-1, (-1, case["group"] or case["n"]))
        scale = (y.abs().amax(-1, keepdim=True) / F8_MAX).clamp(min=TINY)
        res["y8"] = (y / scale).clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn).flatten(-2)
        res["scale"] = scale[..., 0]
    if case["backward"]:
        d = s["dy"].float()
        if z is not None:
            slope = sig * (1 + z * (1 - sig))
            if not case["gate_first"]:
                res["dz"] = (d * m * slope).to(s["x"].dtype)
                d = d * act
        if w is not None:
            res["dw"] = (d * u * r).reshape(-1, case["n"]).sum(0)
            d = d * w
        d = r * (d - u * r * (d * u * r).mean(-1, keepdim=True))
        if z is not None and case["gate_first"]:
            res["dz"] = (d * h * slope).to(s["x"].dtype)
            d = d * act
        if s["dh"] is not None:
            d = d + s["dh"].float()
            res["dresidual"] = d.to(s["residual"].dtype)
        res["dx"] = d.to(s["x"].dtype)
    return res


# ------------------------------------------------------------------------------ one pass

def run(state):
    s, case = state, state["case"]
    if not own:
        return {"gla": _plain_gla, "rms": _plain_rms}[s["op"]](s)
    from state_summary_scan_gb300 import api
    if s["op"] == "gla":
        if case["mode"] == "prefill":
            o = api.gla_prefill(s["plan"], s["q"], s["k"], s["v"], s["g"], s["state"], s["cu"], slots=s["slots"], fresh=s["fresh"])
        else:
            o = api.gla_decode(s["plan"], s["q"], s["k"], s["v"], s["g"], s["state"], slots=s["slots"], fresh=s["fresh"])
        return {"o": o, "state": s["state"]}
    res = {}
    if case["group"] >= 0:
        res["y8"], res["scale"], res["h"] = api.rms_norm_quant(s["x"], s["w"], residual=s["residual"], gate=s["z"],
                                                               gate_first=case["gate_first"], group=case["group"], eps=1e-6)
    else:
        res["y"], res["h"] = api.rms_norm(s["x"], s["w"], residual=s["residual"], gate=s["z"], gate_first=case["gate_first"], eps=1e-6)
    if case["backward"]:
        h = s["x"] if s["residual"] is None else res["h"]
        dx, dresidual, dz, dw = api.rms_norm_backward(h, s["dy"], s["w"], dh=s["dh"], gate=s["z"], gate_first=case["gate_first"], eps=1e-6)
        res["dx"] = dx
        if s["dh"] is not None:
            res["dresidual"] = dresidual
        if s["z"] is not None:
            res["dz"] = dz
        if s["w"] is not None:
            res["dw"] = dw
    if s["residual"] is None:
        del res["h"]
    return res


# ------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "gla":
        S, H, Dk, Dv = case["S"], case["H"], case["Dk"], case["Dv"]
        lens = _lens(case) if case["mode"] == "prefill" else [case["n"]] * S
        N, live = sum(lens), sum(n > 0 for n in lens)
        fresh = sum(n > 0 for n in lens[::2]) if case["fresh"] else 0
        b = N * (2 * case["Hqk"] * Dk + 2 * H * Dv) * SIZE[case["dtype"]] + (2 * live - fresh) * H * Dk * Dv * SIZE[case["state"]]
        b += N * H * 4 if case["gate"] == "token" else H * 4
        return {"bytes": b, "flops": N * H * Dk * Dv * 5}
    rows = case["N"] * case["H"]
    x, e = rows * case["n"], SIZE[case["dtype"]]
    r = SIZE.get(case["residual"], 0)
    b = x * (e + 2 * r)  # x, the residual and their sum
    b += x * e if case["gate"] else 0
    b += x * e if case["group"] < 0 else x + 4 * rows * (case["n"] // case["group"] if case["group"] else 1)
    if case["backward"]:  # dy, dh and the gradients of x, the residual (where it is not that of x) and the gate
        b += x * (2 * e + r + (r if r != e else 0) + (e if case["gate"] else 0))
    return {"bytes": b, "flops": x * (5 + 6 * case["gate"]) * (3 if case["backward"] else 1)}


# ------------------------------------------------------------------------------ the definition in 64 bits

def _exact_gla(s):
    """Each sequence by itself, in blocks: with b the running sum of a block's gates and S the state before it,
    o_t = e^b_t S^T q_t + sum over r <= t of e^(b_t - b_r) (q_t . k_r) v_r."""
    case = s["case"]
    H, ratio = case["H"], case["H"] // case["Hqk"]
    flat = (lambda x: x) if case["mode"] == "prefill" else (lambda x: x.flatten(0, 1))
    q, k, v = (flat(s[x]).double().transpose(0, 1) for x in ("q", "k", "v"))  # [H, N, ...]
    q, k = q.repeat_interleave(ratio, 0) * s["scale"], k.repeat_interleave(ratio, 0)
    g = flat(s["g"]).double().t() if case["gate"] == "token" else s["g"].double()[:, None].expand(H, q.shape[1])
    o, pool, begin = torch.empty_like(v), s["state"].double(), 0
    fresh = s["fresh"].tolist() if s["fresh"] is not None else [0] * case["S"]
    for i, (n, slot) in enumerate(zip(s["lens"], s["slots"].tolist())):
        S = torch.zeros_like(pool[slot]) if fresh[i] else pool[slot]
        for t in range(begin, begin + n, 128):
            at = slice(t, min(t + 128, begin + n))
            qt, kt, vt, b = q[:, at], k[:, at], v[:, at], g[:, at].cumsum(1)
            scores = (qt @ kt.mT) * (b[:, :, None] - b[:, None]).tril().exp().tril()
            o[:, at] = b.exp()[..., None] * (qt @ S) + scores @ vt
            S = S * b[:, -1:, None].exp() + (kt * (b[:, -1:] - b).exp()[..., None]).mT @ vt
        pool[slot] = S
        begin += n
    o = o.transpose(0, 1)
    return {"o": o if case["mode"] == "prefill" else o.unflatten(0, (case["S"], case["n"])), "state": pool}


def _exact_rms(s):
    case = s["case"]
    leaf = lambda t: None if t is None else t.double().requires_grad_(case["backward"])  # noqa: E731
    x, w, z = leaf(s["x"]), leaf(s["w"]), leaf(s["z"])
    res, h = {}, x
    if s["residual"] is not None:
        res["h"] = s["x"].double() + s["residual"].double()
        h = leaf(res["h"].to(s["residual"].dtype))  # as it is kept
    u = h * torch.nn.functional.silu(z) if case["gate_first"] else h
    y = u / (u.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
    y = y if w is None else y * w
    if z is not None and not case["gate_first"]:
        y = y * torch.nn.functional.silu(z)
    if case["group"] < 0:
        res["y"] = y.detach()
    else:
        part = y.detach().unflatten(-1, (-1, case["group"] or case["n"]))
        scale = (part.abs().amax(-1, keepdim=True) / F8_MAX).clamp(min=TINY)
        res["y8"], res["scale"] = (part / scale).flatten(-2), scale[..., 0]
    if case["backward"]:
        names, of = zip(*[(a, b) for a, b in (("dx", h), ("dw", w), ("dz", z)) if b is not None])
        res.update(zip(names, torch.autograd.grad(y, of, s["dy"].double())))
        if s["dh"] is not None:
            res["dresidual"] = res["dx"] = res["dx"] + s["dh"].double()
    return res


def exact(case, seed):
    s = prepare(case, seed)
    return {"gla": _exact_gla, "rms": _exact_rms}[s["op"]](s)
