"""The linear attention block of examples/, its operators together: gradients reach every parameter and agree with
differences, and serving by prefill and decoding gives the training forward's outputs."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "linear_attention_layer.py")
    spec = importlib.util.spec_from_file_location("linear_attention_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_a_step_of_training(example):
    block = example.Block(width=256, heads=2, max_positions=512)
    losses = example.train(block, steps=3)
    assert len(losses) == 3 and all(x == x for x in losses)


def test_the_blocks_gradients_against_differences(example):
    """One direction through every parameter.  bf16 activations leave some 2^-8 of noise in each of the two losses, so the
    step is one that moves the loss by far more than that, and the quotient's own curvature is a few per cent."""
    block = example.Block(width=256, heads=2, max_positions=512, seed=3)
    gen = torch.Generator("cuda").manual_seed(5)
    x, stream, c = (torch.randn(2, 256, 256, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3))

    def loss():
        return (block.train_forward(x, stream, num_segments=4)[0].float() * c.float()).sum()

    grads = torch.autograd.grad(loss(), block.parameters())
    assert all(bool(g.isfinite().all()) and bool((g != 0).any()) for g in grads)
    size = torch.stack([g.square().sum() for g in grads]).sum().sqrt()
    step = 0.05
    values = []
    with torch.no_grad():
        for sign in (1, -2):
            for p, g in zip(block.parameters(), grads):
                p += sign * step * g / size
            values.append(float(loss()))
    got = (values[0] - values[1]) / (2 * step)
    assert abs(got - float(size)) <= 0.1 * float(size)


@pytest.mark.parametrize("eight_bits", [False, True])
def test_serving_is_the_training_forward(example, eight_bits):
    """Every tensor of the path is rounded to bf16 (half a step 2^-8 of it each): eight roundings in a row between the two
    forms, in norm some sqrt(8) 2^-8 = 1.1e-2 at most; in 8 bits two tensors are rounded by 2^-4 / sqrt 3 each in norm."""
    block = example.Block(width=256, heads=2, max_positions=512, seed=4)
    for x, stream, y in zip(*example.serve(block, eight_bits=eight_bits)):
        want = example.trained_outputs(block, x, stream).float()
        limit = 1.2e-2 + (2 ** 0.5 * 2.0 ** -4 / 3 ** 0.5 if eight_bits else 0)
        assert float((y.float() - want).norm() / want.norm()) <= limit
