"""Which device and stream the calls around the mixer launch on, with stand-ins for the library and the GPUs (no GPU)."""
import contextlib

import pytest
import torch

from state_summary_scan_gb300 import _capi as C


class Tensor:
    def __init__(self, device):
        self.device_index = device

    def get_device(self):
        return self.device_index

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def gpus(monkeypatch):
    """Two GPUs of which 0 is current; calls record the device that is current when they are made."""
    now, seen = [0], []

    @contextlib.contextmanager
    def device(d):
        before, now[0] = now[0], d
        yield
        now[0] = before

    class Library:
        def rm_cp_clip_grad_norm(self, *a):
            seen.append((now[0], a[-1]))
            return 0

        def rm_cp_last_error(self):
            return b"no"

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1000 + d, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(C, "_lib", Library())
    monkeypatch.setattr(C, "_by_address", {n: lambda *a: seen.append((now[0], a[-1])) for n in
                                           ("rm_cp_qkr_forward", "rm_cp_qkr_backward", "rm_gdr_state_forward")})
    return now, seen


@pytest.mark.parametrize("where", [0, 1])
def test_calls_launch_on_the_device_of_their_tensors(gpus, where):
    now, seen = gpus
    t, s = Tensor(where), C._raw_stream(None, where)
    C.rm_cp_qkr_forward(1, t, t, t, t, None, None, t, t, s)
    C.rm_cp_qkr_backward(1, t, t, None, None, t, t, t, t, t, t, None, None, None, s)
    C.rm_gdr_state_forward(1, t, t, t, t, t, None, None, None, t, t, t, s)
    C.rm_cp_clip_grad_norm(1, 2, 3, 4, None, None, 0.0, 1e-6, t, t, s)
    assert seen == [(where, 1000 + where)] * 4
    assert now == [0]


def test_a_failed_call_on_another_device_gives_the_current_one_back(gpus, monkeypatch):
    now, _ = gpus
    t = Tensor(1)
    monkeypatch.setitem(C._by_address, "rm_gdr_state_forward", lambda *a: 6)
    with pytest.raises(C.RmCpError):
        C.rm_gdr_state_forward(1, t, t, t, t, t, None, None, None, t, t, t, 0)
    assert now == [0]


def test_a_stream_of_another_device_is_refused(monkeypatch):
    class Stream:
        device_index, cuda_stream = 1, 77

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    assert C._raw_stream(Stream(), 1) == 77
    with pytest.raises(ValueError):
        C._raw_stream(Stream(), 0)
