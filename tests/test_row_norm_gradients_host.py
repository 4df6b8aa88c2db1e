"""The gradients that the norm's adapter passes on (no GPU: the calls are replaced)."""
import pytest
import torch

from state_summary_scan_gb300 import row_norm


@pytest.mark.parametrize("offset", [0, 3, 8])
@pytest.mark.parametrize("residual", [False, True])
def test_gradients_that_autograd_hands_over_unaligned_are_copied(offset, residual, monkeypatch):
    """The gradient of a part of a concatenation is a contiguous view at any offset; the kernels take 16 bytes at a time."""
    seen = []
    monkeypatch.setattr(row_norm, "rms_norm", lambda x, w, r, z, **how: (x * 2, x if r is None else x + r))

    def backward(h, dy, weight, dh, gate, **how):
        seen.extend(t for t in (dy, dh) if t is not None)
        return dy, dy, None, None

    monkeypatch.setattr(row_norm, "rms_norm_backward", backward)
    x = torch.randn(4, 64, requires_grad=True)
    head, weights = torch.zeros(offset), torch.randn(offset + 256)
    got = row_norm.RmsNorm.apply(x, None, torch.randn(4, 64) if residual else None, None, False, 1e-6)
    outs = got if residual else (got,)
    sum((torch.cat([head, y.flatten()]) * weights).sum() for y in outs).backward()
    assert len(seen) == len(outs)
    for t in seen:
        assert t.is_contiguous() and t.data_ptr() % 16 == 0 and torch.equal(t.flatten(), weights[offset:])
