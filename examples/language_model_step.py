"""Data-parallel training steps of a small language model with tied weights, from token numbers to updated weights.

N virtual ranks share one GPU. Each step, every rank looks up its tokens' rows (scaled, with learned positions added by a
second lookup), runs residual blocks of layer norm and two linear layers, and takes the loss straight from the last
norm's output and the table: the logits are never stored. The loss's backward pass writes the table's gradient into its
place in the rank's flat gradient buffer, and the lookup's backward pass adds to it there. The buffers are averaged by the
bucketed ring all-reduce, the norm is clipped on the device, and AdamW steps the fp32 master weights and writes the bf16
weights along. The host reads nothing back but the loss it prints.

    python examples/language_model_step.py [--ranks 4] [--steps 30] [--width 512] [--depth 2] [--vocab 5003]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from ring_all_reduce_02_gb300 import ra  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
PADDING, IGNORE = 0, -100  # the token that fills a sequence up, and the target of a position without a loss


class Model:
    """Tied table and positions, depth x [x = x + W2 relu(W1 norm(x))], a norm; gradients written out by hand."""

    def __init__(self, vocab: int, positions: int, width: int, depth: int, seed: int):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.positions, self.width, self.depth, self.scale = vocab, positions, width, depth, width ** 0.5
        self.shapes = [(vocab, width), (positions, width)]
        for _ in range(depth):
            self.shapes += [(width,), (width,), (2 * width, width), (width, 2 * width)]
        self.shapes += [(width,), (width,)]
        self.counts = [torch.Size(s).numel() for s in self.shapes]
        self.total = sum(self.counts)
        self.master = torch.empty(self.total, device="cuda")
        self.weights = torch.empty(self.total, dtype=BF16, device="cuda")  # what forward and backward use
        for i, (t, s) in enumerate(zip(self.cut(self.master), self.shapes)):
            if len(s) == 2:
                t.copy_(torch.randn(s, generator=gen, device="cuda") * (0.02 if i < 2 else s[1] ** -0.5))
        for norm in range(2, 2 + 4 * depth + 1, 4):  # a norm's weight and bias start a block, and end the model
            self.cut(self.master)[norm].fill_(1.0)
            self.cut(self.master)[norm + 1].zero_()
        self.weights.copy_(self.master)

    def cut(self, flat):
        """The tensors' views of a flat buffer."""
        return [v.view(s) for v, s in zip(flat.split(self.counts), self.shapes)]

    def loss_and_gradients(self, tokens, targets, flat_grads):
        """Mean loss over the positions that have one, of [sequences, positions] tokens and targets; its gradients go
        into ``flat_grads`` (bf16)."""
        w, g = self.cut(self.weights), self.cut(flat_grads)
        sequences, length = tokens.shape
        rows, width, tokens, targets = tokens.numel(), self.width, tokens.reshape(-1), targets.reshape(-1)
        places = torch.arange(length, device="cuda").repeat(sequences)

        def floats(n):
            return torch.empty(n, device="cuda")

        def scratch(n):
            return torch.empty(n, dtype=torch.uint8, device="cuda")

        x = torch.empty(rows, width, dtype=BF16, device="cuda")
        ra.ra_embedding_forward(w[0], tokens, x, scale=self.scale)
        ra.ra_embedding_forward(w[1], places, x, accumulate=True)
        kept = []
        for i in range(2, 2 + 4 * self.depth, 4):
            h, mean, rstd = torch.empty_like(x), floats(rows), floats(rows)
            ra.ra_layernorm_forward(x, w[i], w[i + 1], h, mean, rstd)
            a = torch.relu(h @ w[i + 2].t())
            kept.append((x, h, mean, rstd, a))
            x = x + a @ w[i + 3].t()
        i = 2 + 4 * self.depth
        h, mean, rstd = torch.empty_like(x), floats(rows), floats(rows)
        ra.ra_layernorm_forward(x, w[i], w[i + 1], h, mean, rstd)

        loss, lse, dh = floats(rows), floats(rows), torch.empty_like(h)
        ra.ra_cross_entropy_forward(h, w[0], targets, loss, lse, ignore=IGNORE, workspace=scratch(ra.ra_cross_entropy_workspace(h, w[0])))
        dloss = (1.0 / (targets != IGNORE).sum()).expand(rows).contiguous()
        ra.ra_cross_entropy_backward(h, w[0], targets, lse, dloss, dh, g[0], ignore=IGNORE,
                                     workspace=scratch(ra.ra_cross_entropy_workspace(h, w[0], backward=True)))
        sums = scratch(ra.ra_layernorm_workspace(rows, width))
        dx = torch.empty_like(x)
        ra.ra_layernorm_backward(dh, x, w[i], mean, rstd, dx, g[i], g[i + 1], workspace=sums)
        for i in reversed(range(2, 2 + 4 * self.depth, 4)):
            x, h, mean, rstd, a = kept.pop()
            g[i + 3].copy_(dx.t() @ a)
            da = (dx @ w[i + 3]) * (a > 0)
            g[i + 2].copy_(da.t() @ h)
            through = torch.empty_like(x)
            ra.ra_layernorm_backward(da @ w[i + 2], x, w[i], mean, rstd, through, g[i], g[i + 1], workspace=sums)
            dx = dx + through
        places_scratch = scratch(ra.ra_embedding_workspace(rows, width, self.positions))
        ra.ra_embedding_backward(dx, places, g[1], workspace=places_scratch)
        ra.ra_embedding_backward(dx, tokens, g[0], scale=self.scale, accumulate=True, padding=PADDING,
                                 workspace=scratch(ra.ra_embedding_workspace(rows, width, self.vocab)))
        return (loss * dloss).sum()


class Trainer:
    def __init__(self, model: Model, ranks: int, max_norm: float = 1.0, weight_decay: float = 0.01):
        self.model, self.max_norm, self.steps = model, max_norm, 0
        self.grads = [torch.empty(model.total, dtype=BF16, device="cuda") for _ in range(ranks)]
        self.buckets = ra.ra_bucket_plan(model.counts, 1 << 20, 2)
        self.norm = torch.zeros(2, device="cuda")  # the norm, and the factor that clips it
        self.workspace = torch.zeros(ra.ra_grad_norm_workspace(), dtype=torch.uint8, device="cuda")
        params, grads = model.cut(model.master), model.cut(self.grads[0])
        decay = [weight_decay if len(s) == 2 else 0.0 for s in model.shapes]
        self.list = ra.grad_tensors([self.grads[0]])
        self.tensors = ra.adamw_tensors(params, grads, [torch.zeros_like(p) for p in params], [torch.zeros_like(p) for p in params],
                                        weight_decay=decay, copies=model.cut(model.weights))

    def step(self, batches, lr: float):
        """One step on one (tokens, targets) pair per rank; the ranks' mean loss."""
        losses = [self.model.loss_and_gradients(x, y, g) for (x, y), g in zip(batches, self.grads)]
        ra.ra_allreduce_buckets(self.grads, self.grads, self.buckets, "avg")
        ra.ra_grad_norm(self.list, self.max_norm, self.norm, self.workspace)
        self.steps += 1
        ra.ra_adamw(self.tensors, lr=lr, step=self.steps, grad_scale=self.norm[1:], seed=1)
        return torch.stack(losses).mean()


def samples(vocab: int, sequences: int, length: int, gen):
    """Sequences of unequal lengths in which a fixed map gives each token's successor; the rest is padding."""
    tokens = torch.empty(sequences, length + 1, dtype=torch.int64, device="cuda")
    tokens[:, 0] = torch.randint(1, vocab, (sequences,), generator=gen, device="cuda")
    for i in range(length):
        tokens[:, i + 1] = 1 + (tokens[:, i] * 31 + 7) % (vocab - 1)
    ends = torch.randint(length // 2, length + 1, (sequences, 1), generator=gen, device="cuda")
    there = torch.arange(length, device="cuda") < ends
    return torch.where(there, tokens[:, :-1], PADDING), torch.where(there, tokens[:, 1:], IGNORE)


def train(ranks=4, steps=30, width=512, depth=2, vocab=5003, sequences=8, length=64, lr=2e-3, show=None):
    model = Model(vocab, length, width, depth, seed=0)
    trainer = Trainer(model, ranks)
    gen = torch.Generator(device="cuda").manual_seed(7)
    losses = []
    for k in range(steps):
        loss = trainer.step([samples(vocab, sequences, length, gen) for _ in range(ranks)], lr)
        losses.append(loss)
        if show and (k % 5 == 0 or k == steps - 1):
            show(f"step {k + 1:4d}  loss {float(loss):.5f}  gradient norm {float(trainer.norm[0]):.4f}")
    return [float(v) for v in losses]


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--ranks", type=int, default=4)
    p.add_argument("--steps", type=int, default=30)
    p.add_argument("--width", type=int, default=512)
    p.add_argument("--depth", type=int, default=2)
    p.add_argument("--vocab", type=int, default=5003)
    args = p.parse_args()
    train(args.ranks, args.steps, args.width, args.depth, args.vocab, show=print)
