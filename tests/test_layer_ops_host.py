"""Host-side checks (no GPU) of the per-head norm with rotation, the delta rule with a carried
state, and gradient clipping: refusals before any CUDA call, workspace sizes, and the rotation
table's values."""
import ctypes
import math

import pytest
import torch

from state_summary_scan_gb300 import _capi as C
from state_summary_scan_gb300 import api

A = 1 << 20  # an aligned address that no refused call may touch


def qkr(**kw):
    d = dict(B=2, T=8, Hq=4, Hk=2, D=64, R=32, norm=1, interleaved=0, eps=1e-6, dtype=1, max_pos=64, pos_rows=0, pos64=0)
    strides = dict(q_stride=(2048, 256, 64), k_stride=(1024, 128, 64))
    strides.update({k: kw.pop(k) for k in list(kw) if k in strides})
    d.update(kw)
    return C.QkrProblem(*d.values(), strides["q_stride"], strides["k_stride"])


def status(fn, *args):
    return int(getattr(C.load(), fn)(*args))


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(Hk=0), 1), (dict(dtype=5), 1), (dict(norm=3), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(R=33), 1), (dict(R=66), 1), (dict(R=-2), 1), (dict(max_pos=0), 1), (dict(pos_rows=3), 1),
    (dict(D=60, R=0), 4), (dict(D=264), 4), (dict(q_stride=(2048, 256, 63)), 3), (dict(k_stride=(1024, 129, 64)), 3),
    (dict(k_stride=(-1024, 128, 64)), 1), (dict(B=1 << 16, T=1 << 15), 2),
])
def test_qkr_refuses_bad_problems(kw, want):
    p = qkr(**kw)
    assert status("rm_cp_qkr_forward", p, A, A, None, None, A, None, A, A, None) == want
    assert status("rm_cp_qkr_backward", p, A, A, None, None, A, None, A, A, A, A, None, None, None, None) == want
    assert C.rm_cp_qkr_workspace_size(p) == 0


@pytest.mark.parametrize("at,ptr,want", [(0, None, 1), (1, A + 8, 3), (2, A + 4, 3), (4, None, 1), (6, None, 1), (7, A + 2, 3)])
def test_qkr_refuses_bad_pointers(at, ptr, want):
    args = [A, A, A, A, A, None, A, A]
    args[at] = ptr
    assert status("rm_cp_qkr_forward", qkr(), *args, None) == want


def test_qkr_refuses_missing_positions_and_weights():
    assert status("rm_cp_qkr_forward", qkr(pos_rows=1), A, A, None, None, A, None, A, A, None) == 1
    assert status("rm_cp_qkr_forward", qkr(pos_rows=1, pos64=1), A, A, None, None, A, A + 4, A, A, None) == 3
    # a weight's gradient without the weight, then without a workspace
    assert status("rm_cp_qkr_backward", qkr(), A, A, None, A, A, None, A, A, A, A, A, None, A, None) == 1
    assert status("rm_cp_qkr_backward", qkr(), A, A, A, A, A, None, A, A, A, A, A, None, None, None) == 1


def gds(**kw):
    d = dict(num_seqs=3, num_tokens=12, max_len=8, H=4, qk_heads=2, Dk=64, Dv=64, num_slots=5, scale=0.125, dtype=1, state_dtype=0)
    s = dict(q_stride=(128, 64), k_stride=(128, 64), v_stride=(256, 64), g_stride=4, beta_stride=4)
    s.update({k: kw.pop(k) for k in list(kw) if k in s})
    d.update(kw)
    return C.GdrStateProblem(*d.values(), *s.values())


@pytest.mark.parametrize("kw,want", [
    (dict(num_seqs=0), 1), (dict(num_tokens=-1), 1), (dict(max_len=-1), 1), (dict(H=0), 1), (dict(qk_heads=3), 1), (dict(num_slots=0), 1),
    (dict(dtype=2), 1), (dict(state_dtype=9), 1), (dict(scale=float("inf")), 1), (dict(Dk=48), 4), (dict(Dk=256), 4), (dict(Dv=12), 4),
    (dict(Dv=264), 4), (dict(num_seqs=70000), 2), (dict(q_stride=(129, 64)), 3), (dict(v_stride=(256, 60)), 3), (dict(k_stride=(-8, 64)), 1),
    (dict(g_stride=-1), 1),
])
def test_gdr_state_refuses_bad_problems(kw, want):
    p = gds(**kw)
    assert status("rm_gdr_state_forward", p, A, A, A, A, A, A, A, A, A, A, A, None) == want
    assert C.rm_gdr_state_workspace_size(p) == 0
    assert C.rm_gdr_state_path(p) == -1


@pytest.mark.parametrize("at,ptr,want", [(0, None, 1), (1, A + 8, 3), (2, None, 1), (3, A + 2, 3), (4, None, 1), (5, A + 2, 3), (6, A + 1, 3),
                                         (8, None, 1), (9, A + 8, 3)])
def test_gdr_state_refuses_bad_pointers(at, ptr, want):
    args = [A] * 11
    args[at] = ptr
    assert status("rm_gdr_state_forward", gds(), *args, None) == want


def test_gdr_state_refuses_uneven_and_too_many_sequences():
    none = [None] * 3
    assert status("rm_gdr_state_forward", gds(num_tokens=13), A, A, A, A, A, *none, A, A, A, None) == 2
    assert status("rm_gdr_state_forward", gds(max_len=3), A, A, A, A, A, *none, A, A, A, None) == 2
    assert status("rm_gdr_state_forward", gds(num_slots=2), A, A, A, A, A, *none, A, A, A, None) == 2


def clip(grads=(A, A), numels=(4, 4), dtypes=(0, 1), outs=(A, A), out_dtypes=(0, 1), n=None, max_norm=1.0, eps=1e-6, norm=A, ws=A):
    arr = lambda t, x: None if x is None else (t * len(x))(*x)  # noqa: E731
    return status("rm_cp_clip_grad_norm", len(grads) if n is None else n, arr(ctypes.c_void_p, grads), arr(ctypes.c_int64, numels),
                  arr(ctypes.c_int32, dtypes), arr(ctypes.c_void_p, outs), arr(ctypes.c_int32, out_dtypes), max_norm, eps, norm, ws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=0), 1), (dict(numels=None), 1), (dict(dtypes=None), 1), (dict(out_dtypes=None), 1), (dict(numels=(4, -1)), 1),
    (dict(dtypes=(0, 3)), 1), (dict(out_dtypes=(7, 1)), 1), (dict(grads=(A, None)), 1), (dict(outs=(None, A)), 1),
    (dict(grads=(A + 2, A)), 3), (dict(outs=(A, A + 1)), 3), (dict(out_dtypes=(1, 1)), 1), (dict(max_norm=-1.0), 1),
    (dict(max_norm=float("inf")), 1), (dict(max_norm=float("nan")), 1), (dict(eps=-1.0), 1), (dict(norm=None), 1), (dict(norm=A + 2), 3),
    (dict(ws=None), 1), (dict(numels=(1 << 50, 4)), 2),
])
def test_clip_refuses(kw, want):
    assert clip(**kw) == want


def test_clip_workspace_grows_with_the_tensors():
    assert C.rm_cp_clip_workspace_size(0) == 0
    one, many = C.rm_cp_clip_workspace_size(1), C.rm_cp_clip_workspace_size(5000)
    assert 0 < one < many


def test_cpu_tensors_are_refused():
    with pytest.raises(ValueError):
        api.qk_norm_rope(torch.zeros(1, 2, 4, 64), torch.zeros(1, 2, 4, 64))


def test_rope_table():
    t = api.make_rope_table(50, 8, device="cpu")
    assert t.shape == (50, 2, 4) and t.dtype == torch.float32
    for p in (0, 1, 49):
        for i in range(4):
            a = p * 10000.0 ** (-2 * i / 8)
            assert abs(float(t[p, 0, i]) - math.cos(a)) < 6e-8 and abs(float(t[p, 1, i]) - math.sin(a)) < 6e-8
    # linear: position 4 p of the stretched table is position p
    s = api.make_rope_table(200, 8, scaling="linear", factor=4.0, device="cpu")
    assert torch.equal(s[::4], t)
    # ntk: the fastest pair as before, the slowest as with linear scaling
    n = api.make_rope_table(200, 8, scaling="ntk", factor=4.0, device="cpu")
    assert torch.equal(n[:50, :, 0], t[:, :, 0])
    assert torch.allclose(n[:, :, 3], s[:, :, 3], atol=1e-7)
    # yarn: pairs that turn often are kept, slow ones divided, both scaled
    y = api.make_rope_table(200, 8, scaling="yarn", factor=4.0, trained_positions=400, device="cpu")
    m = 0.1 * math.log(4.0) + 1.0
    assert torch.allclose(y[:50, :, 0], t[:, :, 0] * m, atol=2e-7)
    assert torch.allclose(y[:, :, 3], s[:, :, 3] * m, atol=2e-7)
    for bad in (dict(rotary_dim=7), dict(scaling="other"), dict(factor=0.5), dict(scaling="yarn"), dict(max_positions=0)):
        with pytest.raises(ValueError):
            api.make_rope_table(**{**dict(max_positions=4, rotary_dim=8, device="cpu"), **bad})
