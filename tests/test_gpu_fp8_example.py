"""The example block's training: the loss falls in every step, and each of its four weights'
gradients lowers it alone.  The recorded run of 12 steps goes from 0.714 to 0.038, and one
step of a single weight takes the loss to 0.45 (wg), 0.47 (wu), 0.45 (wd), 0.51 (norm)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(fp4):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_block.py")
    spec = importlib.util.spec_from_file_location("fp8_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_loss_falls_in_every_step(example):
    losses, block, _ = example.train(steps=12)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    assert losses[-1] < 0.1 * losses[0], losses
    start = example.Block(block.M, block.K, block.F, 1)
    for n, w in block.w.items():
        assert not torch.equal(w, start.w[n]), n
    assert not torch.equal(block.norm, start.norm)


@pytest.mark.parametrize("name", ["wg", "wu", "wd", "norm"])
def test_each_gradient_lowers_the_loss_alone(example, name):
    block, target = example.Block(512, 512, 1024, 1), example.Block(512, 512, 1024, 101)
    gen = torch.Generator(device="cuda").manual_seed(201)
    x, r = (torch.randn(512, 512, generator=gen, device="cuda").bfloat16() for _ in range(2))
    want = target.forward(x, r).float()

    def loss():
        diff = block.forward(x, r).float() - want
        return diff, float(diff.square().mean())

    diff, first = loss()
    block.backward((diff * (2.0 / diff.numel())).bfloat16())
    if name == "norm":
        block.norm.sub_(block.dnorm, alpha=60.0)
    else:
        block.w[name].sub_(block.grad[name].float(), alpha=60.0)
        block.quantize_weights()
    assert loss()[1] < 0.85 * first
