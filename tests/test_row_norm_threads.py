"""A call of a norm keeps its checked problem while the C call runs, whatever other threads' calls push out of the cache
(no GPU: the C calls are replaced)."""
import gc
import weakref

import pytest
import torch

from state_summary_scan_gb300 import _capi as C
from state_summary_scan_gb300 import row_norm


@pytest.mark.parametrize("call", ["rms_norm", "rms_norm_quant", "rms_norm_backward"])
def test_a_problem_outlives_its_place_in_the_cache(call, monkeypatch):
    made, alive = [], []

    def checked(x, *args):
        p = C.RmsProblem(4, 1, 64, 1e-6, C.RM_BF16, C.RM_BF16)
        made.append(weakref.ref(p))
        return p

    def pushed_out():  # as 256 other signatures do
        row_norm._CACHE.clear()
        gc.collect()

    def c_call(at, *args):
        pushed_out()
        alive.append(made[-1]() is not None)

    monkeypatch.setattr(row_norm, "_CACHE", type(row_norm._CACHE)())
    monkeypatch.setattr(row_norm, "_checked_problem", checked)
    monkeypatch.setattr(C, "_raw_stream", lambda stream, device: 0)
    for name in ("rm_cp_rms_forward", "rm_cp_rms_quant", "rm_cp_rms_backward"):
        monkeypatch.setattr(C, name, c_call)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    getattr(row_norm, call)(*[x] * (2 if call == "rms_norm_backward" else 1))
    assert alive == [True]
