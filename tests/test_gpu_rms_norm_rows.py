"""Norms of rows: gradients as autograd hands them over, gates far from 0, and more rows than a
launch takes at once."""
import pytest
import test_gpu_rms_norm as one_pass
import torch
from test_gpu_rms_norm import BF, F32, U, close, d, forward64, make

from state_summary_scan_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,res,gate", [(BF, BF, False), (BF, F32, False), (F32, None, False), (BF, None, True)])
def test_parts_of_a_concatenation(dtype, res, gate):
    """The gradient of a concatenation's part starts at any element: the same gradients as of the part alone."""
    x = make((5, 128), dtype, res, gate, seed=4)
    leaves = {k: t.clone().requires_grad_(True) for k, t in x.items() if t is not None}
    y, h = api.rms_norm_train(leaves["x"], leaves["w"], leaves.get("res"), leaves.get("z"))
    g = torch.Generator().manual_seed(2)
    parts = [t for t in (y, h) if t is not leaves["x"]]
    weights = [torch.randn(3 + t.numel(), generator=g).to(t.dtype).cuda() for t in parts]

    def grads(joined):
        def loss(t, w):
            return ((torch.cat([torch.zeros(3, dtype=t.dtype, device="cuda"), t.flatten()]) * w) if joined else (t.flatten() * w[3:])).float().sum()

        return torch.autograd.grad(sum(loss(t, w) for t, w in zip(parts, weights)), list(leaves.values()), retain_graph=True)

    assert all(torch.equal(a, b) for a, b in zip(grads(True), grads(False)))


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("N,n", [(300, 64), (40, 1000), (9, 8192)])
def test_wide_gates_of_fp32_rows(N, n, first):
    """Gates far from 0: their error does not grow with them.  With u = 2^-24: e = e^-|z| is off by 2 u, e / (1 + e) by 7 u, one
    less it by less, silu by 8 u; the slope s (1 + z (1 - s)) by 9 u of itself and 8 u of s |z| (1 - s).  The rest of
    the limits is as in test_gpu_rms_norm.py; a gate before the norm enters the gradients' sums four times."""
    x = make((N, n), F32, gate=True, seed=N)
    g = torch.Generator().manual_seed(n)
    x["z"] = ((torch.rand(N, n, generator=g) * 2 - 1) * 80).cuda()
    dy = torch.randn(N, n, generator=g).cuda()
    y, _ = api.rms_norm(x["x"], x["w"], gate=x["z"], gate_first=first)
    want = forward64(d(x["x"]), d(x["w"]), d(x["z"]), first)
    close(y, want, want.abs() * ((n / 16 + 14 + 1 + 8 + 16 * first) * U), "y")
    dx, _, dz, dw = api.rms_norm_backward(x["x"], dy, x["w"], gate=x["z"], gate_first=first)
    h64, w64, z64 = (d(x[k]).requires_grad_(True) for k in ("x", "w", "z"))
    wx, ww, wz = torch.autograd.grad(forward64(h64, w64, z64, first), (h64, w64, z64), d(dy))
    h, w, z = d(x["x"]), d(x["w"]), d(x["z"])
    s = 1 / (1 + (-z).exp())
    act, mixed = z * s, s * z.abs() * (1 / (1 + z.exp()))
    slope = s * (1 + z * (1 / (1 + z.exp())))
    u = h * act if first else h
    r = 1 / (u.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
    e = d(dy) if first else d(dy) * act
    A = (e * w).abs() * r + u.abs() * r * r * (e * w * u * r).abs().mean(-1, keepdim=True)
    rel = (n / 8 + 40 + 40) * U
    close(dx, wx, rel * (A * act.abs() if first else A) + U * wx.abs() + 1e-44, "dx")
    size = A * h.abs() if first else (u * r * w * d(dy)).abs()
    close(dz, wz, size * (rel * slope.abs() + 8 * U * mixed) + U * wz.abs() + 1e-44, "dgate")
    close(dw, ww, (N / 256 + n / 8 + 64 + 40) * U * (e * u * r).abs().sum(0), "dweight")


# Rows a block takes one after another: a launch has 152 times the blocks that a multiprocessor holds (for rows of 128 a block takes
# 16 at once), so each of these goes round several times, the last one not full.

@pytest.mark.parametrize("N,n,dtype,res,gate,first,dh", [
    (2500, 2048, BF, BF, False, False, True), (2500, 2048, BF, F32, False, False, True), (2500, 2048, F32, F32, False, False, True),
    (2500, 1000, BF, None, False, False, False), (1301, 4096, BF, BF, False, False, True), (1301, 4096, BF, None, True, True, False),
    (401, 8192, BF, BF, False, False, True), (401, 8192, BF, None, True, False, False), (331, 16384, BF, F32, False, False, True),
    (311, 16384, F32, None, True, True, False), (20011, 128, BF, BF, False, False, True), (20011, 128, BF, None, True, False, False),
    (20011, 128, BF, None, True, True, False), (20011, 128, F32, None, True, False, False), (20011, 128, F32, None, True, True, False),
    (40009, 64, BF, None, True, False, False), (10007, 256, BF, F32, False, False, True)])
def test_gradients_of_many_rows(N, n, dtype, res, gate, first, dh):
    one_pass.test_gradients(N, n, dtype, res, gate, first, dh)


@pytest.mark.parametrize("N,H,n,dtype,first", [(1300, 16, 128, BF, False), (1300, 16, 128, F32, True), (2501, 3, 256, BF, True), (700, 2, 2048, BF, False)])
def test_gated_norm_of_many_rows(N, H, n, dtype, first):
    one_pass.test_gated_norm_of_slices(N, H, n, dtype, first)


@pytest.mark.parametrize("N,n,res,gate,first,group", [(20011, 128, None, True, False, 32), (20011, 128, None, True, True, 0), (1301, 4096, BF, False, False, 128),
                                                      (811, 8192, BF, False, False, 0), (331, 16384, None, False, False, 64)])
def test_eight_bits_of_many_rows(N, n, res, gate, first, group):
    """Row by row the bits that calls of a few rows give (which are tested against the formula)."""
    x = make((N, n), BF, res, gate, seed=N)
    y8, scale, h = api.rms_norm_quant(x["x"], x["w"], residual=x["res"], gate=x["z"], gate_first=first, group=group)
    part = lambda t, at: None if t is None else t[at: at + 100]  # noqa: E731
    for at in range(0, N, 100):
        few = api.rms_norm_quant(part(x["x"], at), x["w"], residual=part(x["res"], at), gate=part(x["z"], at), gate_first=first, group=group)
        assert all(torch.equal(a.view(torch.uint8), part(b, at).contiguous().view(torch.uint8)) for a, b in zip(few, (y8, scale, h)))
