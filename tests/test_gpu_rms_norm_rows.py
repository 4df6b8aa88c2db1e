"""Norms of rows: gradients as autograd hands them over."""
import pytest
import torch
from test_gpu_rms_norm import BF, F32, make

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
