"""The example layer: training lowers the loss, and serving gives what the training forward gives."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("delta_rule_layer", os.path.join(ROOT, "examples", "delta_rule_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_trains_and_serves():
    m = load()
    layer = m.Layer(width=128, heads=2, max_positions=1024)
    losses = m.train(layer, steps=12, T=256)
    assert all(a > 0 for a in losses) and losses[-1] < losses[0]
    xs, outs = m.serve(layer, lens=(70, 5, 64), generate=3)
    for x, y in zip(xs, outs):
        n = x.shape[0]
        padded = torch.cat([x, torch.zeros(256 - n, 128, dtype=x.dtype, device="cuda")])
        with torch.no_grad():
            want = layer.train_forward(padded[None], num_segments=4)[0, :n]
        # both forms in bf16 with other roundings: the framework's tolerance for bf16 storage
        assert float((y.float() - want.float()).abs().max()) <= 2e-2 * float(want.float().abs().max())
