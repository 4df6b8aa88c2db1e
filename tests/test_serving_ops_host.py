"""Host-side checks (no GPU) of linear attention on a pool of states and of the norms of rows: refusals before any CUDA
call, workspace sizes, how rows are found in strided tensors, and the devices that the calls launch on."""
import pytest
import torch
from test_layer_ops_devices import Tensor, gpus  # noqa: F401
from test_layer_ops_host import A, gds, status

from state_summary_scan_gb300 import _capi as C
from state_summary_scan_gb300 import api, row_norm


@pytest.mark.parametrize("kw,want", [
    (dict(num_seqs=0), 1), (dict(num_tokens=-1), 1), (dict(H=0), 1), (dict(qk_heads=3), 1), (dict(num_slots=0), 1), (dict(dtype=2), 1),
    (dict(scale=float("nan")), 1), (dict(Dk=48), 4), (dict(Dk=256), 4), (dict(Dv=12), 4), (dict(Dv=264), 4), (dict(num_seqs=70000), 2),
    (dict(q_stride=(129, 64)), 3), (dict(k_stride=(-8, 64)), 1), (dict(g_stride=-1), 1),
])
def test_gla_state_refuses_bad_problems(kw, want):
    p = gds(**kw)
    assert status("rm_cp_gla_state_forward", p, *[A] * 10, None) == want
    assert C.rm_cp_gla_state_workspace_size(p) == 0 and C.rm_cp_gla_state_path(p) == -1


@pytest.mark.parametrize("at,ptr,want", [(0, None, 1), (1, A + 8, 3), (2, None, 1), (3, A + 2, 3), (4, A + 2, 3), (5, A + 1, 3), (7, None, 1), (8, A + 8, 3)])
def test_gla_state_refuses_bad_pointers(at, ptr, want):
    args = [A] * 10
    args[at] = ptr
    assert status("rm_cp_gla_state_forward", gds(), *args, None) == want


def test_gla_state_refuses_uneven_and_too_many_sequences():
    none = [None] * 3
    assert status("rm_cp_gla_state_forward", gds(num_tokens=13), A, A, A, A, *none, A, A, A, None) == 2
    assert status("rm_cp_gla_state_forward", gds(max_len=3), A, A, A, A, *none, A, A, A, None) == 2
    assert status("rm_cp_gla_state_forward", gds(num_slots=2), A, A, A, A, *none, A, A, A, None) == 2


@pytest.mark.parametrize("kw,want", [
    (dict(), 0), (dict(num_tokens=4000, max_len=4000), 1), (dict(num_tokens=4000, max_len=63), 0), (dict(num_tokens=4000, max_len=4000, dtype=0, q_stride=(128, 64)), 0),
    (dict(num_tokens=400, max_len=32, Dk=128, q_stride=(256, 128), k_stride=(256, 128)), 1), (dict(num_tokens=31, max_len=400, Dk=128, q_stride=(256, 128), k_stride=(256, 128)), 0),
    (dict(num_tokens=4000, max_len=4000, Dk=32, q_stride=(64, 32), k_stride=(64, 32)), 0),
])
def test_gla_state_paths(kw, want):
    p = gds(**kw)
    assert C.rm_cp_gla_state_path(p) == want
    assert C.rm_cp_gla_state_workspace_size(p) >= 16
    if want:  # one that keeps to the recurrence
        p.recurrent = 1
        assert C.rm_cp_gla_state_path(p) == 0


def rms(**kw):
    d = dict(N=4, H=2, n=64, eps=1e-6, dtype=1, res_dtype=1, gate=0, group=0)
    s = dict(x_stride=(128, 64), r_stride=(128, 64), z_stride=(128, 64))
    s.update({k: kw.pop(k) for k in list(kw) if k in s})
    d.update(kw)
    return C.RmsProblem(*d.values(), *s.values())


def at(i):  # addresses far apart
    return A + (i << 24)


def forward(p, x=at(0), res=None, z=None, w=None, h=None, y=at(5)):
    return status("rm_cp_rms_forward", p, x, res, z, w, h, y, None)


def quant(p, x=at(0), res=None, z=None, w=None, h=None, y=at(5), s=at(6)):
    return status("rm_cp_rms_quant", p, x, res, z, w, h, y, s, None)


def backward(p, h=at(0), z=None, w=None, dy=at(1), dh=None, dx=at(2), dr=None, dz=None, dw=None, ws=None):
    return status("rm_cp_rms_backward", p, h, z, w, dy, dh, dx, dr, dz, dw, ws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), 1), (dict(H=0), 1), (dict(n=0), 1), (dict(dtype=2), 1), (dict(res_dtype=7), 1), (dict(dtype=0), 4), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(gate=3), 1), (dict(n=60), 4), (dict(n=32776), 4), (dict(group=16), 4), (dict(group=128), 2), (dict(N=1 << 16, H=1 << 15), 2),
    (dict(x_stride=(-128, 64)), 1), (dict(x_stride=(100, 64)), 3), (dict(r_stride=(128, 63)), 3), (dict(z_stride=(4, 64)), 3),
])
def test_rms_refuses_bad_problems(kw, want):
    p = rms(**kw)
    assert forward(p) == want and quant(p) == want and backward(p) == want
    assert C.rm_cp_rms_workspace_size(p) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), 1), (dict(x=at(0) + 8), 3), (dict(y=None), 1), (dict(y=at(5) + 4), 3), (dict(w=at(3) + 4), 3), (dict(res=at(1)), 1), (dict(res=at(1) + 2, h=at(2)), 3),
    (dict(res=at(1), h=at(2) + 8), 3),
    # overlaps: y within x, h on x, h within the residual, y on the weight, y on h
    (dict(y=at(0) + 128), 1), (dict(res=at(1), h=at(0)), 1), (dict(res=at(1), h=at(1) + 256), 1), (dict(w=at(5) + 64), 1), (dict(res=at(1), h=at(5)), 1),
])
def test_rms_forward_refuses_bad_tensors(kw, want):
    assert forward(rms(), **kw) == want


def test_rms_forward_refuses_a_gate_beside_a_residual_and_without_its_tensor():
    assert forward(rms(gate=1), res=at(1), h=at(2), z=at(3)) == 4
    assert forward(rms(gate=2)) == 1
    assert quant(rms(), s=None) == 1 and quant(rms(), s=at(6) + 2) == 3
    assert quant(rms(), y=at(0)) == 1  # 8 bits over x
    assert quant(rms(), s=at(5) + 16) == 1


@pytest.mark.parametrize("p,kw,want", [
    ({}, dict(h=None), 1), ({}, dict(dy=at(1) + 4), 3), ({}, dict(dx=None), 1), ({}, dict(dw=at(5)), 1), ({}, dict(w=at(4), dw=at(5)), 1),
    ({}, dict(w=at(4), dw=at(5), ws=at(6) + 8), 3), (dict(gate=1), dict(z=at(3)), 1), (dict(gate=1), dict(dz=at(3)), 1), (dict(gate=1), dict(z=at(3), dz=at(4), dh=at(5)), 4),
    (dict(res_dtype=0), {}, 1), ({}, dict(dx=at(1) + 64), 1), ({}, dict(w=at(4), dw=at(4), ws=at(6)), 1), (dict(gate=1), dict(z=at(3), dz=at(2)), 1),
    ({}, dict(w=at(4), dw=at(5), ws=at(2)), 1),
])
def test_rms_backward_refuses_bad_tensors(p, kw, want):
    assert backward(rms(**p), **kw) == want


def test_rms_workspace_holds_the_partial_gradients():
    sizes = [C.rm_cp_rms_workspace_size(rms(N=1, H=1, n=n)) for n in (8, 128, 256, 1000, 4096, 32768)]
    assert all(s > 0 and s % 16 == 0 for s in sizes)


def test_cpu_tensors_are_refused():
    x = torch.zeros(2, 64)
    for call in (api.rms_norm, api.rms_norm_quant):
        with pytest.raises(ValueError):
            call(x)
    with pytest.raises(ValueError):
        api.rms_norm_backward(x, x)


@pytest.mark.parametrize("shape,take,want", [
    ((5, 64), lambda t: t, (5, 1, [(64, 0)])), ((5, 3, 64), lambda t: t, (15, 1, [(64, 0)])), ((5, 3, 64), lambda t: t[:, 1:], (5, 2, [(192, 64)])),
    ((5, 3, 64), lambda t: t.transpose(0, 1), (3, 5, [(64, 192)])), ((2, 5, 3, 64), lambda t: t[:, :, :2], (10, 2, [(192, 64)])),
    ((2, 5, 3, 64), lambda t: t[:, :4, :2], None), ((64,), lambda t: t, (1, 1, [(0, 0)])), ((1, 7, 1, 64), lambda t: t, (7, 1, [(64, 0)])),
])
def test_rows_of_strided_tensors(shape, take, want):
    t = take(torch.zeros(shape))
    if want is None:
        with pytest.raises(ValueError):
            row_norm._rows([t])
        return
    N, H, strides = row_norm._rows([t])
    assert N * H == t.numel() // t.shape[-1]
    flat = t.as_strided((N, H, 64), (*strides[0], 1))
    u = torch.arange(t.numel()).view(t.shape)
    assert (N, H, strides) == want
    t.copy_(u)
    assert torch.equal(flat.reshape(-1), u.reshape(-1).float())


def test_rows_of_two_tensors_are_found_together():
    x, z = torch.zeros(6, 4, 32), torch.zeros(6, 4, 96)[..., :32]
    assert row_norm._rows([x, z]) == (24, 1, [(32, 0), (96, 0)])
    z = torch.zeros(6, 5, 32)[:, :4]
    assert row_norm._rows([x, z]) == (6, 4, [(128, 32), (160, 32)])


@pytest.mark.parametrize("where", [0, 1])
def test_calls_launch_on_the_device_of_their_tensors(gpus, where, monkeypatch):  # noqa: F811
    now, seen = gpus
    for n in ("rm_cp_gla_state_forward", "rm_cp_rms_forward", "rm_cp_rms_quant", "rm_cp_rms_backward"):
        monkeypatch.setitem(C._by_address, n, lambda *a: seen.append((now[0], a[-1])))
    t, s = Tensor(where), C._raw_stream(None, where)
    C.rm_cp_gla_state_forward(1, t, t, t, t, None, None, None, t, t, t, s)
    C.rm_cp_rms_forward(1, t, None, None, None, None, t, s)
    C.rm_cp_rms_quant(1, t, t, None, t, t, t, t, s)
    C.rm_cp_rms_backward(1, t, None, None, t, None, t, t, None, None, None, s)
    assert seen == [(where, 1000 + where)] * 4
    assert now == [0]


def offsets(rows):
    N, H, (step,) = rows
    return [i * step[0] + j * step[1] for i in range(N) for j in range(H)]


@pytest.mark.parametrize("base,shape", [((2, 1, 64), (2, 3, 64)), ((4, 1, 64), (4, 5, 64)), ((1, 3, 64), (2, 3, 64)), ((1, 64), (3, 64)), ((64,), (2, 3, 64)),
                                        ((2, 1, 1, 64), (2, 3, 5, 64)), ((1, 3, 1, 64), (2, 3, 5, 64))])
def test_rows_of_broadcast_tensors_stay_in_them(base, shape):
    x = torch.zeros(base).expand(shape)
    want = [int(i) for i in torch.arange(x.untyped_storage().size() // 4).reshape(base).expand(shape)[..., 0].flatten()]
    try:
        got = row_norm._rows([x])
    except ValueError:
        assert base == (1, 3, 1, 64)  # two broadcast dimensions around another: three steps
    else:
        assert offsets(got) == want


@pytest.mark.parametrize("shape", [(0, 64), (3, 0, 64), (0, 3, 64), (3, 0, 2, 64)])
def test_tensors_without_rows_have_no_tokens(shape):
    assert row_norm._rows([torch.zeros(shape)])[0] == 0


def test_gla_state_refuses_outputs_and_states_over_other_tensors():
    p = gds()  # q, k, v, g, cu_seqlens, slots, fresh, state, o, ws
    args = [at(i) for i in range(10)]
    for out, over in [(8, 0), (8, 1), (8, 2), (8, 3), (8, 7), (7, 0), (7, 1), (7, 2), (7, 3)]:
        for shift in (0, 16):
            bad = list(args)
            bad[out] = args[over] + shift
            assert status("rm_cp_gla_state_forward", p, *bad, None) == 1, (out, over, shift)
            assert b"overlap" in C.load().rm_cp_last_error()
