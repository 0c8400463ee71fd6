"""examples/language_model_step.py: lookup, norms, loss and their gradients together, as a training program uses them."""

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
    spec = importlib.util.spec_from_file_location("language_model_step", os.path.join(ROOT, "examples", "language_model_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("ranks,width,vocab", [(2, 128, 1000), (3, 72, 257)])
def test_runs(example, ranks, width, vocab):
    losses = example.train(ranks=ranks, steps=4, width=width, depth=1, vocab=vocab, sequences=3, length=40)
    assert len(losses) == 4 and all(v == v for v in losses)
    # an untrained model's loss: log(vocab) of uniform words, and half the logits' variance. They are a norm's output
    # (length sqrt(width)) times the table's 0.02: a variance of width 0.02^2 = 0.05 at most
    assert abs(losses[0] - torch.tensor(float(vocab)).log().item()) < 0.1


@pytest.mark.parametrize("width,vocab", [(128, 500), (100, 333)])
def test_gradients_match_autograd(example, width, vocab, monkeypatch):
    # the hand-written backward pass in bf16 against autograd in 64 bits on the same weights. Every activation and
    # gradient passes a few bf16 roundings (2^-9 each) per layer on its way, each of them independent: in the 2-norm
    # 12 stages of 3 roundings are off by about sqrt(36) 2^-9 = 1.2%; 4% is allowed. The units that are on are the run's own:
    # roundings of about 2^-9 sqrt(3) of a unit's input, which is of variance 1, flip its sign in one of 1000, and a share p
    # of flipped units is off by sqrt(2 p) = 4.5% in the 2-norm, twice with two blocks, though neither side is wrong.
    length, depth = 24, 2
    model = example.Model(vocab, length, width, depth, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(5)
    tokens, targets = example.samples(vocab, 10, length, gen)
    flat = torch.empty(model.total, dtype=torch.bfloat16, device="cuda")
    on, relu = [], torch.relu
    monkeypatch.setattr(torch, "relu", lambda x: on.append(x > 0) or relu(x))
    loss = model.loss_and_gradients(tokens, targets, flat)
    monkeypatch.undo()
    assert len(on) == depth
    w = [t.double().requires_grad_() for t in model.cut(model.weights)]
    functional = torch.nn.functional
    h = functional.embedding(tokens, w[0], padding_idx=example.PADDING) * model.scale + w[1]
    for i, mask in zip(range(2, 2 + 4 * depth, 4), on):
        units = functional.layer_norm(h, (width,), w[i], w[i + 1], 1e-5) @ w[i + 2].t()
        h = h + (units * mask.view(*tokens.shape, -1)) @ w[i + 3].t()
    i = 2 + 4 * depth
    out = functional.layer_norm(h, (width,), w[i], w[i + 1], 1e-5) @ w[0].t()
    want = functional.cross_entropy(out.reshape(-1, vocab), targets.reshape(-1), ignore_index=example.IGNORE)
    want.backward()
    value = float(want.detach())
    assert abs(float(loss) - value) <= 0.02 * value
    for got, t in zip(model.cut(flat), w):
        assert float((got.double() - t.grad).norm()) <= 0.04 * float(t.grad.norm())


def test_ranks_average(example):
    # two ranks with the same samples step as one rank does: the average of equal gradients is exact
    a = example.train(ranks=1, steps=3, width=64, depth=1, vocab=300, sequences=4, length=32)
    model = example.Model(300, 32, 64, 1, seed=0)
    trainer = example.Trainer(model, 2)
    gen = torch.Generator(device="cuda").manual_seed(7)
    b = []
    for _ in range(3):
        batch = example.samples(300, 4, 32, gen)
        b.append(float(trainer.step([batch, batch], 2e-3)))
    assert a == b
