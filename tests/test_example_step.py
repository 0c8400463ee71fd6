"""examples/data_parallel_step.py: the operators together, as a training program uses them."""

import importlib.util
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from ring_all_reduce_02_gb300 import build

    build.build()
    spec = importlib.util.spec_from_file_location("data_parallel_step", os.path.join(ROOT, "examples", "data_parallel_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("moments", ["f32", "8bit"])
@pytest.mark.parametrize("ranks,width", [(4, 256), (3, 200)])
def test_loss_falls(example, moments, ranks, width):
    losses = example.train(ranks=ranks, steps=25, moments=moments, width=width, depth=2, rows=512)
    assert all(v == v for v in losses)
    assert losses[-1] < 0.5 * losses[0], losses


def test_gradients_match_autograd(example):
    # the hand-written backward pass in bf16 against autograd in 64 bits on the same weights. Every activation and
    # gradient passes a few bf16 roundings (2^-9 each) per layer on its way, each of them independent: in the 2-norm
    # 12 stages of 3 roundings are off by about sqrt(36) 2^-9 = 1.2%; 4% is allowed.
    model = example.Model(256, 2, 32, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, y = example.samples(256, 32, 300, gen)
    flat = torch.empty(model.total, dtype=torch.bfloat16, device="cuda")
    loss = model.loss_and_gradients(x, y, flat)
    w = [t.double().requires_grad_() for t in model.cut(model.weights)]
    h = x.double()
    norm = torch.nn.functional.layer_norm
    for i in range(0, 8, 4):
        h = h + torch.relu(norm(h, (256,), w[i], w[i + 1], 1e-5) @ w[i + 2].t()) @ w[i + 3].t()
    out = norm(h, (256,), w[8], w[9], 1e-5) @ w[10].t()
    want = (out - y.double()).square().mean()
    want.backward()
    value = float(want.detach())
    assert abs(float(loss) - value) <= 0.02 * value
    for got, t in zip(model.cut(flat), w):
        assert float((got.double() - t.grad).norm()) <= 0.04 * float(t.grad.norm())


def test_ranks_average(example):
    # two ranks with the same samples step as one rank does: the average of equal gradients is exact
    a = example.train(ranks=1, steps=3, width=128, depth=1, rows=64)
    model = example.Model(128, 1, 64, seed=0)
    trainer = example.Trainer(model, 2, "f32")
    gen = torch.Generator(device="cuda").manual_seed(7)
    b = []
    for _ in range(3):
        batch = example.samples(128, 64, 64, gen)
        b.append(float(trainer.step([batch, batch], 2e-3)))
    assert a == b
