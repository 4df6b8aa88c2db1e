"""Norms of rows against their formulas in 64 bits, and gradients against the formula's and differences.

Limits, element by element, with u = 2^-24 (fp32), w = half a step of the output's type (bf16 2^-8, e4m3 2^-4):
  a row's sum of squares is off by at most (n / 8 + 16) u of itself in the worst order of additions, its root by half of
  that; each y takes six roundings more: |y| ((n / 16 + 14) u + w).  silu is off by 8 u and the argument of its
  exponential by |z| u.
  Gradients are sums of two terms of sizes A and B: ((n / 8 + 32) u (A + B)) + w |value|; a weight's gradient adds N rows,
  (N / 256 + n / 8 + 64) u of the absolute sum (a block adds its own rows in turn, then the blocks' sums eight at a time)."""
import math

import pytest
import torch

from state_summary_scan_gb300 import api

pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24
EPS = 1e-6


def half(dtype):
    return {F32: 2.0 ** -24, BF: 2.0 ** -8, F8: 2.0 ** -4}[dtype]


def make(shape, dtype, res=None, gate=False, weight=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = dict(x=rnd(*shape).to(dtype), res=None, z=None, w=None)
    if res is not None:
        big = 1 + 40 * (torch.rand(shape[-1], generator=g) < 0.02)
        x["res"] = (3 * rnd(*shape) * big).to(res)
    if gate:
        x["z"] = (2 * rnd(*shape)).to(dtype)
    if weight:
        x["w"] = 1 + 0.3 * rnd(shape[-1])
    return {k: None if t is None else t.cuda() for k, t in x.items()}


def forward64(h, w, z, first):
    """y of the rows h, all in 64 bits"""
    act = None if z is None else z / (1 + (-z).exp())
    u = h * act if first else h
    y = u / (u.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
    y = y if w is None else y * w
    return y if act is None or first else y * act


def d(t):
    return None if t is None else t.detach().double().cpu()


def close(got, want, far, name):
    err = (d(got) - want).abs()
    ok = err <= far
    assert bool(ok.all()), f"{name}: {float((err / far)[~ok].max()):.2f} of its limit"


def y_limit(y, n, z, dtype):
    return y.abs() * ((n / 16 + 14) * U + half(dtype) + (0 if z is None else (8 + z.abs()) * U)) + 1e-30


LENGTHS = [8, 64, 72, 128, 136, 256, 264, 1000, 1024, 2048, 2056, 4096, 5120, 8192, 8200, 16384, 32768]


@pytest.mark.parametrize("dtype,res", [(BF, None), (BF, BF), (BF, F32), (F32, None), (F32, F32)])
@pytest.mark.parametrize("n", LENGTHS)
@pytest.mark.parametrize("N", [1, 7, 331])
def test_norm(N, n, dtype, res):
    x = make((N, n), dtype, res, weight=n != 1000, seed=n + N)
    y, h = api.rms_norm(x["x"], x["w"], residual=x["res"])
    h64 = d(x["x"]) if res is None else d(x["x"]) + d(x["res"])
    if res is not None:
        assert h.dtype == res
        close(h, h64, h64.abs() * (half(res) + U) + 1e-30, "h")
        h64 = d(h)
    else:
        assert h is x["x"]
    want = forward64(h64, d(x["w"]), None, False)
    close(y, want, y_limit(want, n, None, dtype), "y")


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,H,n", [(1, 1, 64), (61, 16, 128), (5, 3, 96), (33, 2, 256), (9, 1, 2048), (3, 2, 4104), (2, 1, 8192), (2, 1, 16384)])
def test_gated_norm_of_slices(N, H, n, dtype, first):
    x = make((N, H, n), dtype, gate=True, seed=n)
    wide = torch.full((N, 3 * H * n), float("nan"), dtype=dtype, device="cuda")  # a projection: the other slices are not read
    wide[:, H * n: 2 * H * n] = x["z"].flatten(1)
    z = wide[:, H * n: 2 * H * n].unflatten(-1, (H, n))
    y, _ = api.rms_norm(x["x"], x["w"], gate=z, gate_first=first)
    want = forward64(d(x["x"]), d(x["w"]), d(x["z"]), first)
    # gate first: the activation's error is in the row's sum too
    extra = (10 + d(x["z"]).abs().max()) * U * 2 if first else 0.0
    close(y, want, y_limit(want, n, d(x["z"]), dtype) + want.abs() * extra, "y")


@pytest.mark.parametrize("dtype,res,gate,first", [(BF, BF, False, False), (BF, F32, False, False), (F32, None, False, False), (BF, None, True, False),
                                                  (F32, None, True, True)])
@pytest.mark.parametrize("n,group", [(64, 0), (64, 32), (64, 64), (96, 32), (128, 64), (128, 128), (256, 128), (1024, 32), (2048, 0), (2056, 0), (4096, 128), (8192, 64),
                                     (16384, 128)])
def test_eight_bits(n, group, dtype, res, gate, first):
    N = 19
    x = make((N, n), dtype, res, gate, seed=n + group)
    x["x"][3] = 0  # a row of zeros: its scale is the smallest, its values are 0
    if res is not None:
        x["res"][3] = 0
    y8, scale, h = api.rms_norm_quant(x["x"], x["w"], residual=x["res"], gate=x["z"], gate_first=first, group=group)
    assert y8.dtype == F8 and scale.shape == (N, n // (group or n))
    want = forward64(d(h), d(x["w"]), d(x["z"]), first).unflatten(-1, (-1, group or n))
    top = want.abs().amax(-1)
    s64 = (top / 448).clamp(min=2.0 ** -126)
    rel = (n / 16 + 24) * U + (0 if x["z"] is None else 3 * (10 + float(d(x["z"]).abs().max())) * U)
    close(scale, s64, s64 * rel, "scale")
    got = d(y8).unflatten(-1, (-1, group or n)) * d(scale)[..., None]
    # half a step of e4m3: 2^-4 of the value, or half of the smallest step, 2^-10, of the scale
    close(got, want, want.abs() * (2.0 ** -4 + 2 * rel) + s64[..., None] * (2.0 ** -10 + 448 * rel), "y8")
    assert bool((d(y8)[3] == 0).all()) and float(scale[3].max()) == 2.0 ** -126
    assert float(d(y8).abs().max()) <= 448


@pytest.mark.parametrize("dtype,res,gate,first,dh", [(BF, BF, False, False, True), (BF, F32, False, False, True), (BF, None, False, False, False),
                                                     (F32, F32, False, False, True), (F32, F32, False, False, False), (BF, None, True, False, False),
                                                     (BF, None, True, True, False), (F32, None, True, False, False), (F32, None, True, True, False)])
@pytest.mark.parametrize("N,n", [(1, 64), (700, 128), (41, 256), (300, 1000), (5, 2048), (40, 4096), (3, 5120), (7, 8192), (3, 16384)])
def test_gradients(N, n, dtype, res, gate, first, dh):
    x = make((N, n), dtype, res, gate, weight=n != 256, seed=N + n)
    g = torch.Generator().manual_seed(N)
    dy = torch.randn(N, n, generator=g).to(dtype).cuda()
    up = torch.randn(N, n, generator=g).to(res or dtype).cuda() if dh else None
    h = x["x"] if res is None else api.rms_norm(x["x"], x["w"], residual=x["res"])[1]
    dx, dres, dz, dw = api.rms_norm_backward(h, dy, x["w"], dh=up, gate=x["z"], gate_first=first)
    leaf = lambda t: None if t is None else d(t).requires_grad_(True)  # noqa: E731
    h64, w64, z64 = leaf(h), leaf(x["w"]), leaf(x["z"])
    y = forward64(h64, w64, z64, first)
    wanted = [t for t in (h64, w64, z64) if t is not None]
    grads = dict(zip([id(t) for t in wanted], torch.autograd.grad(y, wanted, d(dy))))
    # sizes of the terms: e w r, and u r times the mean
    z, w = d(x["z"]), d(x["w"])
    act = None if z is None else z / (1 + (-z).exp())
    u = d(h) * act if first else d(h)
    r = 1 / (u.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
    e = d(dy) if act is None or first else d(dy) * act
    ew = e if w is None else e * w
    A = ew.abs() * r + u.abs() * r * r * (ew * u * r).abs().mean(-1, keepdim=True)
    rel = (n / 8 + 40) * U + (0 if z is None else 4 * (10 + float(z.abs().max())) * U)
    slope = None if z is None else (1 / (1 + (-z).exp())) * (1 + z * (1 - 1 / (1 + (-z).exp())))
    want = grads[id(h64)]
    far = rel * (A if not first else A * act.abs())
    if up is not None:
        want = want + d(up)
        far = far + 2 * U * (want.abs() + d(up).abs())
    close(dx, want, far + half(dtype) * want.abs() + 1e-30, "dx")
    assert dres.dtype == h.dtype
    close(dres, want, far + half(h.dtype) * want.abs() + 1e-30, "dresidual")
    if z is not None:
        want = grads[id(z64)]
        size = (u * r).abs() * (1 if w is None else w.abs()) * d(dy).abs() if not first else A * d(h).abs()
        # the slope is 1 at its largest, and its own sum loses what its two terms have in common
        far = 2 * rel * size * (slope.abs() + (1 + z.abs()) * 2.0 ** -20) + rel * size
        close(dz, want, far + half(dtype) * want.abs() + 1e-30, "dgate")
    if w is not None:
        size = (e * u * r).abs().sum(0)
        close(dw, grads[id(w64)], (N / 256 + n / 8 + 64 + (0 if z is None else 60)) * U * size + 1e-30, "dweight")


@pytest.mark.parametrize("res,gate,first", [(F32, False, False), (None, True, False), (None, True, True)])
def test_gradients_against_differences(res, gate, first):
    """Central differences of the formula in 64 bits along one direction: off by the third derivative, some 1e-6."""
    x = make((4, 64), F32, res, gate, seed=8)
    leaves = {k: t.clone().requires_grad_(True) for k, t in x.items() if t is not None}
    y, h = api.rms_norm_train(leaves["x"], leaves["w"], leaves.get("res"), leaves.get("z"), gate_first=first)
    g = torch.Generator().manual_seed(3)
    a, b = (torch.randn(4, 64, generator=g, dtype=torch.float64) for _ in range(2))
    loss = (y.double().cpu() * a).sum() + ((h.double().cpu() * b).sum() if res is not None else 0)
    loss.backward()
    way = {k: torch.randn(t.shape, generator=g, dtype=torch.float64) for k, t in leaves.items()}

    def value(step):
        p = {k: d(t) + step * way[k] for k, t in leaves.items()}
        h64 = p["x"] + p["res"] if res is not None else p["x"]
        return float((forward64(h64, p["w"], p.get("z"), first) * a).sum() + ((h64 * b).sum() if res is not None else 0))

    want = (value(1e-4) - value(-1e-4)) / 2e-4
    got = sum(float((d(t.grad) * way[k]).sum()) for k, t in leaves.items())
    size = sum(float((d(t.grad) * way[k]).abs().sum()) for k, t in leaves.items())
    assert abs(got - want) <= 200 * U * size + 1e-5


def test_training_form_uses_and_drops_what_it_gives():
    x = make((6, 2048), BF, BF, seed=5)
    a, r, w = (x[k].clone().requires_grad_(True) for k in ("x", "res", "w"))
    y, h = api.rms_norm_train(a, w, r)
    h.float().sum().backward()  # y is not used: the gradients pass by
    assert bool((a.grad == 1).all()) and bool((r.grad == 1).all()) and w.grad is None
    a.grad = r.grad = None
    y, h = api.rms_norm_train(a, w, r)
    (dx,) = torch.autograd.grad(y.float().square().sum(), a)
    want = api.rms_norm_backward(h.detach(), (2 * y.detach().float()).to(BF), w.detach())[0]
    assert torch.equal(dx, want)
    with pytest.raises(RuntimeError):  # no second derivative
        (dx,) = torch.autograd.grad(api.rms_norm_train(a, w, r)[0].float().square().sum(), a, create_graph=True)
        dx.float().sum().backward()


def test_in_place_and_given_outputs():
    x = make((33, 2048), BF, BF, seed=9)
    want, total = api.rms_norm(x["x"], x["w"], residual=x["res"])
    stream, out = x["res"].clone(), torch.empty_like(x["x"])
    v = stream._version
    y, h = api.rms_norm(x["x"], x["w"], residual=stream, out=out, h=stream)
    assert y is out and h is stream and torch.equal(out, want) and torch.equal(stream, total) and stream._version > v
    same = x["x"].clone()
    y, _ = api.rms_norm(same, x["w"], out=same)
    assert y is same and torch.equal(same, api.rms_norm(x["x"], x["w"])[0])
    y8, s = torch.empty_like(x["x"], dtype=F8), torch.empty(33, 16, device="cuda")
    got = api.rms_norm_quant(x["x"], x["w"], residual=x["res"], group=128, out=(y8, s))
    again = api.rms_norm_quant(x["x"], x["w"], residual=x["res"], group=128)
    assert got[0] is y8 and torch.equal(y8.view(torch.uint8), again[0].view(torch.uint8)) and torch.equal(s, again[1])


def test_layouts():
    """Rows spaced in one or two dimensions; others are refused."""
    g = torch.Generator().manual_seed(1)
    wide = torch.randn(6, 5, 4, 96, generator=g).to(BF).cuda()
    for x in (wide[..., 32:], wide[:, 1], wide[:, :, 2], wide.transpose(0, 1)[:, :, 0], wide[2, 3], wide[2, 3, 1], wide[:, 1:4, 2:3, :64]):
        y, _ = api.rms_norm(x)
        assert y.shape == x.shape and y.is_contiguous() and torch.equal(y, api.rms_norm(x.contiguous())[0])
    with pytest.raises(ValueError):
        api.rms_norm(wide.transpose(0, 2))
    with pytest.raises(ValueError):
        api.rms_norm(wide.transpose(2, 3))


def test_nothing_to_do():
    x = torch.empty(0, 128, dtype=BF, device="cuda")
    w = torch.ones(128, device="cuda")
    assert api.rms_norm(x, w)[0].shape == x.shape
    y8, s, _ = api.rms_norm_quant(x, w, group=64)
    assert y8.shape == x.shape and s.shape == (0, 2)
    dx, _, _, dw = api.rms_norm_backward(x, x, w)
    assert dx.shape == x.shape and bool((dw == 0).all())


def test_infinities_and_nan_stay_in_their_rows():
    x = make((5, 2048), BF, seed=2)
    want = api.rms_norm_quant(x["x"], x["w"], group=128)
    x["x"][1, 7], x["x"][3, 9] = float("nan"), float("inf")
    y, _ = api.rms_norm(x["x"], x["w"])
    assert bool(y[1].isnan().all()) and bool(y[3, 9].isnan()) and bool((y[3, :9] == 0).all())
    y8, s, _ = api.rms_norm_quant(x["x"], x["w"], group=128)
    assert bool(s[1].isnan().all())
    for i in (0, 2, 4):
        assert torch.equal(y8[i].view(torch.uint8), want[0][i].view(torch.uint8)) and torch.equal(s[i], want[1][i])


def test_weight_gradients_do_not_depend_on_the_launch():
    x = make((4099, 128), BF, gate=True, seed=6)
    dy = torch.randn(4099, 128, device="cuda").to(BF)
    first = api.rms_norm_backward(x["x"], dy, x["w"], gate=x["z"])
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(api.rms_norm_backward(x["x"], dy, x["w"], gate=x["z"]), first))


def test_other_streams_and_graphs():
    x = make((257, 4096), BF, BF, seed=4)
    dy = torch.randn(257, 4096, device="cuda").to(BF)
    want = api.rms_norm_quant(x["x"], x["w"], residual=x["res"])
    grads = api.rms_norm_backward(x["res"], dy, x["w"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = api.rms_norm_quant(x["x"], x["w"], residual=x["res"], stream=s)
    back = api.rms_norm_backward(x["res"], dy, x["w"], stream=s)
    s.synchronize()
    assert all(torch.equal(a.float(), b.float()) for a, b in zip(got, want))
    assert torch.equal(back[0], grads[0]) and torch.equal(back[3], grads[3])
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = api.rms_norm_quant(x["x"], x["w"], residual=x["res"])
            back = api.rms_norm_backward(x["res"], dy, x["w"])
    x["x"].mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    want = api.rms_norm_quant(x["x"], x["w"], residual=x["res"])
    assert all(torch.equal(a.float(), b.float()) for a, b in zip(got, want)) and torch.equal(back[0], grads[0])


@pytest.mark.parametrize("change", [
    dict(weight=torch.ones(128)), dict(weight="bf16"), dict(residual="short"), dict(gate="f32"), dict(residual="x", gate="x"), dict(gate_first=True),
    dict(residual="bf16 for f32"),
])
def test_refusals(change):
    x = torch.randn(4, 128, device="cuda").to(BF)
    kw = {k: x if v == "x" else torch.ones(128, device="cuda", dtype=BF) if v == "bf16" else x[:3] if v == "short" else x.float() if v == "f32" else v
          for k, v in change.items()}
    if change.get("residual") == "bf16 for f32":
        x, kw = x.float(), dict(residual=x)
    with pytest.raises(ValueError):
        api.rms_norm(x, **kw)


def test_refused_sizes_and_overlaps():
    from state_summary_scan_gb300 import RmCpError
    x = torch.randn(4, 256, device="cuda").to(BF)
    for bad in (x[:, :100], torch.zeros(1, 32776, device="cuda")):
        with pytest.raises(RmCpError):
            api.rms_norm(bad.contiguous())
    with pytest.raises(RmCpError):
        api.rms_norm_quant(x, group=96)
    with pytest.raises(RmCpError):
        api.rms_norm_quant(x[:, :96].contiguous(), group=64)
    flat = torch.randn(5 * 256, device="cuda").to(BF)
    with pytest.raises(RmCpError):  # y over a part of x
        api.rms_norm(flat[:1024].view(4, 256), out=flat[256:].view(4, 256))
    with pytest.raises(RmCpError):  # h over x
        api.rms_norm(x, residual=x.clone(), h=x)
    with pytest.raises(ValueError):
        api.rms_norm(x, h=x)


@pytest.mark.parametrize("base", [(5, 1, 128), (1, 3, 128), (128,), (5, 1, 1, 128)])
def test_broadcast_inputs(base):
    shape = (5, 3, 128) if len(base) < 4 else (5, 2, 3, 128)
    g = torch.Generator().manual_seed(9)
    one = torch.randn(*base, generator=g).to(BF)
    other = torch.randn(*shape, generator=g).to(BF)
    for x, res in ((one.expand(shape), other), (other, one.expand(shape))):
        y, h = api.rms_norm(x.cuda().expand(shape) if x is other else one.cuda().expand(shape), residual=one.cuda().expand(shape) if res is not other else other.cuda())
        total = (d(x) + d(res)).to(BF)
        assert torch.equal(h.cpu(), total)
        want = forward64(d(total), None, None, False)
        close(y, want, y_limit(want, 128, None, BF), "y")
    z = one.cuda().expand(shape)
    y, _ = api.rms_norm(other.cuda(), gate=z)
    want = forward64(d(other), None, d(z), False)
    close(y, want, y_limit(want, 128, d(z), BF), "gated y")


def test_gradient_of_a_broadcast_input():
    x = torch.randn(5, 1, 128, generator=torch.Generator().manual_seed(3))
    dy = torch.randn(5, 3, 128, generator=torch.Generator().manual_seed(4))
    leaf = x.cuda().requires_grad_()
    y, _ = api.rms_norm_train(leaf.expand(5, 3, 128))
    y.backward(dy.cuda())
    ref = x.double().requires_grad_()
    forward64(ref.expand(5, 3, 128), None, None, False).backward(dy.double())
    r = (ref.detach().pow(2).mean(-1, keepdim=True) + EPS).rsqrt()
    # du = r (d - uh mean(d uh)), three rows added: the limits of a gradient of terms A and B, with two additions more
    uh = ref.detach() * r
    size = (dy.double().abs() * r + uh.abs() * r * (dy.double() * uh).abs().mean(-1, keepdim=True)).sum(1, keepdim=True)
    close(leaf.grad, ref.grad, (128 / 8 + 34) * U * size + half(F32) * ref.grad.abs(), "dx")


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("first", [False, True])
def test_nan_in_a_gate_of_8_bits(first, group):
    x = make((5, 3, 128), BF, gate=True)
    x["z"][2, 1, 70] = float("nan")
    y8, s, _ = api.rms_norm_quant(x["x"], x["w"], gate=x["z"], gate_first=first, group=group)
    back = y8.float() * s.repeat_interleave(group or 128, -1)
    x["z"][2, 1, 70] = 0  # all but the row are as without it
    clean8, cs, _ = api.rms_norm_quant(x["x"], x["w"], gate=x["z"], gate_first=first, group=group)
    rest = torch.ones(5, 3, dtype=torch.bool, device="cuda")
    rest[2, 1] = False
    assert torch.equal(y8.view(torch.uint8)[rest], clean8.view(torch.uint8)[rest]) and torch.equal(s[rest], cs[rest])
    bad = back[2, 1].isnan()
    if first:
        assert bool(bad.all()) and bool(s[2, 1].isnan().all())
    else:
        assert int(bad.sum()) == 1 and bool(bad[70]) and not bool(s.isnan().any())
        assert torch.equal(s, cs)
