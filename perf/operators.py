"""Cases that measure the serving and training operators around the gated recurrences:

  qkr   per-head norm of queries and keys with the position rotation in the same pass
        (forward, and forward + backward)
  gds   the gated delta rule with a carried state: recurrent (a few tokens for each of many
        sequences, state updated in place) and ragged prefill (whole prompts)
  clip  the global norm of many gradient tensors, and clipping

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


# ------------------------------------------------------------------------------ the cases

def _qkr(name, B, T, Hq, Hk, D, R, **kw):
    c = dict(op="qkr", B=B, T=T, Hq=Hq, Hk=Hk, D=D, R=R, norm="rms", weight=True, interleaved=False,
             dtype="bf16", backward=False, fused_qkv=False, max_pos=32768, scaling="none")
    c.update(kw)
    return dict(c, name=name) if name else c


def _gds(name, S, n, H, Hqk, Dk, Dv, **kw):
    # n: tokens of each sequence (decode) or the longest sequence (prefill)
    c = dict(op="gds", mode="decode", S=S, n=n, H=H, Hqk=Hqk, Dk=Dk, Dv=Dv, dtype="bf16", state="f32", lens=0,
             fresh=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def _clip(name, tensors, total, dtype, lens, **kw):
    c = dict(op="clip", tensors=tensors, total=total, dtype=dtype, lens=lens, clip=True)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of each of 32 sequences in decoding, each at its own position: latency
        _qkr("qkr decode", 32, 1, 16, 16, 128, 128),
        # prompts of odd length on slices of a fused projection, few key heads, a quarter of a small
        # head rotated in interleaved pairs, delta-rule style unit keys
        _qkr("qkr prefill odd", 3, 1009, 16, 2, 64, 16, norm="l2", weight=False, interleaved=True, fused_qkv=True),
        # fp32 training step of a small model, positions stretched for a longer context
        _qkr("qkr train fp32", 2, 2047, 8, 8, 64, 64, dtype="f32", backward=True, scaling="linear"),
        # the training step of the 32k configuration
        _qkr("qkr train 32k", 1, 32768, 16, 16, 128, 128, backward=True),
        # one sequence, one token, the 64-wide heads of the 8k configuration: the smallest call
        _gds("gds decode 1", 1, 1, 16, 16, 64, 64),
        # a batch of users, one token each, 128-wide heads, fp32 state
        _gds("gds decode 256", 256, 1, 16, 16, 128, 128),
        # several tokens checked at a time, bf16 state, heads sharing queries and keys, wide values
        _gds("gds decode 4 tokens", 61, 4, 32, 16, 128, 256, state="bf16"),
        # a fp32 model of odd sizes, ragged prompts with an empty and a one-token one
        _gds("gds prefill fp32", 7, 301, 6, 3, 32, 40, mode="prefill", dtype="f32", lens=3),
        # one 8k prompt of 128-wide heads
        _gds("gds prefill 8k", 1, 8192, 16, 16, 128, 128, mode="prefill", state="bf16", fresh=True),
        # ragged prompts of a batch, heads sharing queries and keys, some continuing a state
        _gds("gds prefill ragged", 13, 4096, 32, 16, 128, 128, mode="prefill", state="bf16", lens=5, fresh=True),
        # the gradients of a small model: many small fp32 tensors
        _clip("clip small", 75, 2_000_003, "f32", 1),
        # the gradients of a large model in bf16 and fp32
        _clip("clip large", 311, 805_306_421, "mix", 2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["qkr", "qkr", "decode", "decode", "prefill", "prefill", "clip"])
    if op == "qkr":
        D = rng.choice([32, 64, 80, 96, 128, 128, 256])
        Hk = rng.choice([1, 2, 4, 8, 16])
        Hq = Hk * rng.choice([1, 1, 2, 4]) if Hk <= 8 else Hk
        n = _log(rng, 1, (32768 * 32 * 128) // ((Hq + Hk) * D))
        B = min(n, _log(rng, 1, 64))
        T = max(1, n // B)
        return _qkr(None, B, min(T, 32768), Hq, Hk, D, rng.choice([D, D, D // 2, 16]), norm=rng.choice(["rms", "rms", "l2", "none"]),
                    weight=rng.random() < 0.6, interleaved=rng.random() < 0.4, dtype=rng.choice(["bf16", "bf16", "f32"]) if n < 8192 else "bf16",
                    backward=rng.random() < 0.5, fused_qkv=rng.random() < 0.4, scaling=rng.choice(["none", "none", "linear", "yarn"]))
    if op == "decode":
        Dk, Dv = rng.choice([(64, 64), (128, 128), (128, 256), (32, 48), (128, 64), (64, 128)])
        Hqk = rng.choice([2, 4, 8, 16])
        H = Hqk * rng.choice([1, 2])
        S = _log(rng, 1, max(1, min(512, (256 * 16 * 128 * 128) // (H * Dk * Dv))))
        return _gds(None, S, rng.choice([1, 1, 1, 2, 3, 5, 8]), H, Hqk, Dk, Dv, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    state=rng.choice(["f32", "bf16"]), fresh=rng.random() < 0.3)
    if op == "prefill":
        f32 = rng.random() < 0.3
        S = _log(rng, 1, 16)
        Hqk = rng.choice([2, 4, 8, 16])
        H = Hqk * rng.choice([1, 2]) if Hqk < 16 else 16
        Dk, Dv = rng.choice([(64, 64), (128, 128), (128, 256), (32, 48), (64, 128)])
        most = min(4096, (4096 * 13 * 32 * 128 * 128) // (S * H * Dk * Dv))
        return _gds(None, S, _log(rng, 2, 500 if f32 else most), H, Hqk, Dk, Dv, mode="prefill", dtype="f32" if f32 else "bf16",
                    state="f32" if f32 else "bf16", lens=rng.randrange(1, 1000), fresh=rng.random() < 0.5)
    dtype = rng.choice(["f32", "bf16", "mix"])
    return _clip(None, _log(rng, 1, 400), _log(rng, 1000, 500_000_000 if dtype == "f32" else 700_000_000), dtype, rng.randrange(1000),
                 clip=rng.random() < 0.8)


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


def _numels(case):
    """Sizes of the gradient tensors: many small, some large, odd ones among them; their sum is `total`."""
    r = random.Random(case["lens"])
    n = min(case["tensors"], max(1, case["total"] // 2))
    w = [math.exp(r.gauss(0, 2.2)) for _ in range(n)]
    out = [max(1, int((case["total"] - n) * x / sum(w))) for x in w]
    out[max(range(n), key=lambda i: out[i])] += max(0, case["total"] - sum(out))
    return out


def _clip_types(case, n):
    return [("bf16" if i % 3 else "f32") if case["dtype"] == "mix" else case["dtype"] for i in range(n)]


# ------------------------------------------------------------------------------ the inputs

def _table(case, dev):
    """cos and sin of each position: [max_pos, 2, R/2] fp32, with the scaling of a longer context."""
    R = case["R"]
    i = torch.arange(R // 2, dtype=torch.float64)
    inv, factor, mult = 10000.0 ** (-2 * i / R), 4.0, 1.0
    if case["scaling"] == "linear":
        inv = inv / factor
    elif case["scaling"] == "yarn":
        turns = 8192 * inv / (2 * math.pi)  # turns of a pair over the trained context
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        inv, mult = inv * keep + inv / factor * (1 - keep), 0.1 * math.log(factor) + 1.0
    a = torch.arange(case["max_pos"], dtype=torch.float64)[:, None] * inv
    return (torch.stack([a.cos(), a.sin()], 1) * mult).float().contiguous().to(dev)


def _prepare_qkr(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    B, T, Hq, Hk, D, dt = (case[x] for x in ("B", "T", "Hq", "Hk", "D", "dtype"))
    dt = F[dt]
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    if case["fused_qkv"]:  # queries, keys and values of one projection
        x = (rnd(B, T, (Hq + 2 * Hk) * D) * 2).to(dt)
        q = x[..., : Hq * D].unflatten(-1, (Hq, D))
        k = x[..., Hq * D: (Hq + Hk) * D].unflatten(-1, (Hk, D))
    else:
        q, k = (rnd(B, T, Hq, D) * 2).to(dt), (rnd(B, T, Hk, D) * 2).to(dt)
    first = torch.randint(0, case["max_pos"] - T + 1, (B, 1), generator=g, device=dev)
    s = {"op": "qkr", "case": case, "q": q, "k": k, "table": _table(case, dev),
         "pos": (first + torch.arange(T, device=dev)).to(torch.int32), "wq": None, "wk": None}
    if case["weight"]:
        s["wq"], s["wk"] = 1 + 0.2 * rnd(D), 1 + 0.2 * rnd(D)
    if case["backward"]:
        s["dq"], s["dk"] = rnd(B, T, Hq, D).to(dt), rnd(B, T, Hk, D).to(dt)
    return s


def _prepare_gds(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    S, n, H, Hqk, Dk, Dv = (case[x] for x in ("S", "n", "H", "Hqk", "Dk", "Dv"))
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    prefill = case["mode"] == "prefill"
    lens = _lens(case) if prefill else [n] * S
    N = sum(lens)
    dt, st = F[case["dtype"]], F[case["state"]]
    k = rnd(N, Hqk, Dk)
    k = (k / k.norm(dim=-1, keepdim=True)).to(dt)
    slots = S + 3  # the pool has room for others
    s = {"op": "gds", "case": case, "q": rnd(N, Hqk, Dk).to(dt), "k": k, "v": rnd(N, H, Dv).to(dt),
         "g": torch.nn.functional.logsigmoid(rnd(N, H) + 4), "beta": torch.sigmoid(rnd(N, H)),
         "state": (0.3 * rnd(slots, H, Dk, Dv)).to(st),
         "slots": torch.randperm(slots, generator=g, device=dev)[:S].to(torch.int32),
         "lens": lens, "scale": Dk ** -0.5, "fresh": None}
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    if case["fresh"]:  # every other sequence begins
        s["fresh"] = (torch.arange(S, device=dev) % 2 == 0).to(torch.uint8)
    if not prefill:
        for x in ("q", "k", "v", "g", "beta"):
            s[x] = s[x].unflatten(0, (S, n))
    if own:
        from state_summary_scan_gb300 import api
        s["plan"] = api.make_gdr_state_plan(S, N, H, Dk, Dv, num_slots=slots, qk_heads=Hqk, max_len=max(lens), scale=s["scale"],
                                            dtype=dt, state_dtype=st, device=dev)
    return s


def _prepare_clip(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    sizes = _numels(case)
    types = _clip_types(case, len(sizes))
    flat, out, at = {}, {}, {}
    for t in sorted(set(types)):
        total = sum(n for n, x in zip(sizes, types) if x == t)
        flat[t] = torch.empty(total, dtype=F[t], device=dev).normal_(0, 1e-3, generator=g)
        out[t], at[t] = torch.empty_like(flat[t]), 0
    grads, outs = [], []
    for n, t in zip(sizes, types):
        grads.append(flat[t][at[t]: at[t] + n])
        outs.append(out[t][at[t]: at[t] + n])
        at[t] += n
    s = {"op": "clip", "case": case, "grads": grads, "outs": outs, "flat": out, "max_norm": 1e-3 * math.sqrt(case["total"]) / 2}
    if own:
        from state_summary_scan_gb300 import api
        s["plan"] = api.make_clip_plan(len(grads), device=dev)
    return s


def prepare(case, seed):
    return {"qkr": _prepare_qkr, "gds": _prepare_gds, "clip": _prepare_clip}[case["op"]](case, seed)


# ------------------------------------------------------------------------------ the plain forms

def _pairs(x, R, interleaved):
    """The two members of each rotated pair."""
    return (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., : R // 2], x[..., R // 2: R])


def _join(a, b, rest, interleaved):
    both = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([both, rest], -1)


def _turn(x, c, s, R, interleaved):
    a, b = _pairs(x, R, interleaved)
    return _join(a * c - b * s, b * c + a * s, x[..., R:], interleaved)


def _scale_of(x, norm, eps):
    if norm == "none":
        return None
    t = (x * x).sum(-1, keepdim=True)
    return torch.rsqrt((t / x.shape[-1] if norm == "rms" else t) + eps)


def _plain_qkr(s):
    case = s["case"]
    R, inter, norm, eps = case["R"], case["interleaved"], case["norm"], 1e-6
    cs = s["table"][s["pos"].long()][:, :, None]
    c, sn = cs[..., 0, :], cs[..., 1, :]
    res = {}
    for n in ("q", "k"):
        x, w = s[n].float(), s["w" + n]
        r = _scale_of(x, norm, eps)
        y = x if r is None else x * r
        y = y if w is None else y * w
        res[n] = _turn(y, c, sn, R, inter).to(s[n].dtype)
        if case["backward"]:
            d = _turn(s["d" + n].float(), c, -sn, R, inter)  # the rotation's transpose
            h = x if r is None else x * r
            if w is not None:
                res["dw" + n] = (d * h).sum((0, 1, 2))
                d = d * w
            if r is not None:
                m = (d * h).sum(-1, keepdim=True)
                d = r * (d - h * (m / x.shape[-1] if norm == "rms" else m))
            res["d" + n] = d.to(s[n].dtype)
    return res


def _plain_gds(s):
    case = s["case"]
    S, H, Hqk, L = case["S"], case["H"], case["Hqk"], max(s["lens"])
    prefill = case["mode"] == "prefill"
    if prefill:  # padded to the longest: a token past a sequence's end changes nothing
        at = torch.arange(L, device=s["cu"].device)[:, None] + s["cu"][None, :-1]
        live = at < s["cu"][None, 1:]
        at = torch.where(live, at, 0).long()
        get = lambda x: torch.where(live.view(L, S, *[1] * (x.dim() - 1)), x[at].float(), 0.0)  # noqa: E731
    else:
        get = lambda x: x.transpose(0, 1).float()  # noqa: E731
    q, k, v, a, beta = get(s["q"]), get(s["k"]), get(s["v"]), get(s["g"]).exp(), get(s["beta"])
    q, k = q.repeat_interleave(H // Hqk, 2) * s["scale"], k.repeat_interleave(H // Hqk, 2)
    slots = s["slots"].long()
    state = s["state"][slots].float()
    if s["fresh"] is not None:
        state = torch.where(s["fresh"].view(S, 1, 1, 1) != 0, 0.0, state)
    outs = []
    for t in range(L):
        state = state * a[t][..., None, None]
        d = beta[t][..., None] * (v[t] - torch.matmul(k[t][..., None, :], state)[..., 0, :])
        state = state + k[t][..., None] * d[..., None, :]
        outs.append(torch.matmul(q[t][..., None, :], state)[..., 0, :])
    o = torch.stack(outs)
    if prefill:
        o = o.transpose(0, 1)[live.transpose(0, 1)]
    else:
        o = o.transpose(0, 1)
    s["state"][slots] = state.to(s["state"].dtype)
    return {"o": o.to(s["v"].dtype), "state": s["state"]}


def _plain_clip(s):
    total = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    if not s["case"]["clip"]:
        return {"norm": total}
    coef = (s["max_norm"] / (total + 1e-6)).clamp(max=1.0)
    for g, o in zip(s["grads"], s["outs"]):
        o.copy_(g.float() * coef)
    return {"norm": total, "out": s["flat"]}


# ------------------------------------------------------------------------------ one pass

def run(state):
    s, case = state, state["case"]
    if not own:
        return {"qkr": _plain_qkr, "gds": _plain_gds, "clip": _plain_clip}[s["op"]](s)
    from state_summary_scan_gb300 import api
    if s["op"] == "qkr":
        how = dict(positions=s["pos"], q_weight=s["wq"], k_weight=s["wk"], norm=case["norm"], eps=1e-6, interleaved=case["interleaved"])
        q, k = api.qk_norm_rope(s["q"], s["k"], s["table"], **how)
        res = {"q": q, "k": k}
        if case["backward"]:
            dq, dk, dwq, dwk = api.qk_norm_rope_backward(s["q"], s["k"], s["dq"], s["dk"], s["table"], **how)
            res.update(dq=dq, dk=dk)
            if s["wq"] is not None:
                res.update(dwq=dwq, dwk=dwk)
        return res
    if s["op"] == "gds":
        if case["mode"] == "prefill":
            o = api.gdr_prefill(s["plan"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["cu"], slots=s["slots"], fresh=s["fresh"])
        else:
            o = api.gdr_decode(s["plan"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"], fresh=s["fresh"])
        return {"o": o, "state": s["state"]}
    if not case["clip"]:
        return {"norm": api.clip_grad_norm(s["plan"], s["grads"])}
    norm = api.clip_grad_norm(s["plan"], s["grads"], s["max_norm"], out=s["outs"])
    return {"norm": norm, "out": s["flat"]}


# ------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "qkr":
        n = case["B"] * case["T"]
        x = n * (case["Hq"] + case["Hk"]) * case["D"]
        b = x * SIZE[case["dtype"]] * (4 if case["backward"] else 2) + n * 4 + min(n, case["max_pos"]) * case["R"] * 4
        return {"bytes": b, "flops": x * (18 if case["backward"] else 7)}
    if case["op"] == "gds":
        S, H, Dk, Dv = case["S"], case["H"], case["Dk"], case["Dv"]
        lens = _lens(case) if case["mode"] == "prefill" else [case["n"]] * S
        N, live = sum(lens), sum(n > 0 for n in lens)
        fresh = sum(n > 0 for n in lens[::2]) if case["fresh"] else 0
        b = N * (2 * case["Hqk"] * Dk + 2 * H * Dv) * SIZE[case["dtype"]] + N * H * 8 + (2 * live - fresh) * H * Dk * Dv * SIZE[case["state"]]
        return {"bytes": b, "flops": N * H * Dk * Dv * 7}
    sizes = _numels(case)
    b = sum(n * SIZE[t] for n, t in zip(sizes, _clip_types(case, len(sizes))))
    return {"bytes": b * (2 if case["clip"] else 1), "flops": sum(sizes) * (3 if case["clip"] else 2)}


# ------------------------------------------------------------------------------ the definition in 64 bits

def _exact_qkr(s):
    case = s["case"]
    R, D = case["R"], case["D"]
    turn = torch.complex(*s["table"].double()[s["pos"].long()].unbind(2))[:, :, None]  # one factor a pair
    res = {}
    for n in ("q", "k"):
        x = s[n].double().requires_grad_(True)
        w = s["w" + n].double().requires_grad_(True) if s["w" + n] is not None else None
        y = x
        if case["norm"] == "rms":
            y = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
        elif case["norm"] == "l2":
            y = x / (x.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt()
        y = y if w is None else y * w
        z = y[..., :R].unflatten(-1, (R // 2, 2) if case["interleaved"] else (2, R // 2))
        z = torch.complex(z[..., 0], z[..., 1]) if case["interleaved"] else torch.complex(z[..., 0, :], z[..., 1, :])
        z = z * turn
        z = torch.stack([z.real, z.imag], -1 if case["interleaved"] else -2).flatten(-2)
        y = torch.cat([z, y[..., R:]], -1) if R < D else z
        res[n] = y.detach()
        if case["backward"]:
            got = torch.autograd.grad(y, [x] + ([w] if w is not None else []), s["d" + n].double())
            res["d" + n] = got[0]
            if w is not None:
                res["dw" + n] = got[1]
    return res


def _exact_gds(s):
    """In blocks: with b the running gate sum of a block and S the state before it, the written values D solve
    (I + tril(beta k k^T e^(b_t - b_r), -1)) D = beta (v - e^b k S)."""
    case = s["case"]
    r = case["H"] // case["Hqk"]
    flat = (lambda x: x) if case["mode"] == "prefill" else (lambda x: x.flatten(0, 1))
    q, k, v, g, beta = (flat(s[x]).double().transpose(0, 1) for x in ("q", "k", "v", "g", "beta"))  # [H, N, ...]
    q, k = q.repeat_interleave(r, 0) * s["scale"], k.repeat_interleave(r, 0)
    o, pool, begin = torch.empty_like(v), s["state"].double(), 0
    fresh = s["fresh"].tolist() if s["fresh"] is not None else [0] * case["S"]
    for i, (n, slot) in enumerate(zip(s["lens"], s["slots"].tolist())):
        S = torch.zeros_like(pool[slot]) if fresh[i] else pool[slot]
        for t in range(begin, begin + n, 128):
            at = slice(t, min(t + 128, begin + n))
            qt, kt, vt, be, b = q[:, at], k[:, at], v[:, at], beta[:, at, None], g[:, at].cumsum(1)
            gap = (b[:, :, None] - b[:, None]).tril().exp().tril()
            A = (be * (kt @ kt.mT) * gap).tril(-1)
            D = torch.linalg.solve_triangular(A + torch.eye(A.shape[-1], device=A.device, dtype=A.dtype),
                                              be * (vt - (kt * b.exp()[..., None]) @ S), upper=False, unitriangular=True)
            o[:, at] = (qt * b.exp()[..., None]) @ S + ((qt @ kt.mT) * gap) @ D
            S = S * b[:, -1:, None].exp() + (kt * (b[:, -1:] - b).exp()[..., None]).mT @ D
        pool[slot] = S
        begin += n
    o = o.transpose(0, 1)
    return {"o": o if case["mode"] == "prefill" else o.unflatten(0, (case["S"], case["n"])), "state": pool}


def _exact_clip(s):
    norm = math.sqrt(sum(float(g.double().pow(2).sum()) for g in s["grads"]))
    total = torch.tensor(norm, dtype=torch.float64, device=s["grads"][0].device)
    if not s["case"]["clip"]:
        return {"norm": total}
    coef = min(1.0, s["max_norm"] / (norm + 1e-6))
    types = [str(g.dtype) for g in s["grads"]]
    return {"norm": total, "out": {t: torch.cat([g.double() * coef for g, x in zip(s["grads"], types) if x == str(F[t])]) for t in s["flat"]}}


def exact(case, seed):
    s = prepare(case, seed)
    return {"qkr": _exact_qkr, "gds": _exact_gds, "clip": _exact_clip}[s["op"]](s)
