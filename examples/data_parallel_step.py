"""Data-parallel training steps of a small residual model, with every operator of the library in its place.

N virtual ranks share one GPU. Each step, every rank runs forward and backward on its own samples; layer norm's
backward pass writes its weight gradients straight into the rank's flat gradient buffer. The buffers are averaged by
the bucketed ring all-reduce, the gradient norm is measured and turned into the clip factor on the device, and AdamW
steps the fp32 master weights (moments in fp32 or in 8 bits) and writes the bf16 weights along. The host reads nothing
back but the loss it prints.

    python examples/data_parallel_step.py [--ranks 4] [--steps 30] [--moments f32|8bit] [--width 512] [--depth 4]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from ring_all_reduce_02_gb300 import ra  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class Model:
    """depth x [x = x + W2 relu(W1 norm(x))], then a norm and a linear head; gradients written out by hand."""

    def __init__(self, width: int, depth: int, outputs: int, seed: int):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.shapes = []
        for _ in range(depth):
            self.shapes += [(width,), (width,), (2 * width, width), (width, 2 * width)]
        self.shapes += [(width,), (width,), (outputs, width)]
        self.depth = depth
        self.counts = [torch.Size(s).numel() for s in self.shapes]
        self.total = sum(self.counts)
        self.master = torch.empty(self.total, device="cuda")
        self.weights = torch.empty(self.total, dtype=BF16, device="cuda")  # what forward and backward use
        for t, s in zip(self.cut(self.master), self.shapes):
            if len(s) == 2:
                t.copy_(torch.randn(s, generator=gen, device="cuda") * s[1] ** -0.5)
        for norm in range(0, 4 * depth + 1, 4):  # a norm's weight and bias start a block, and end the model
            self.cut(self.master)[norm].fill_(1.0)
            self.cut(self.master)[norm + 1].zero_()
        self.weights.copy_(self.master)

    def cut(self, flat):
        """The tensors' views of a flat buffer."""
        return [v.view(s) for v, s in zip(flat.split(self.counts), self.shapes)]

    def loss_and_gradients(self, x, target, flat_grads):
        """Mean squared error of one rank's samples; its gradients go into ``flat_grads`` (bf16)."""
        w, g = self.cut(self.weights), self.cut(flat_grads)
        rows, width = x.shape
        scratch = torch.empty(ra.ra_layernorm_workspace(rows, width), dtype=torch.uint8, device="cuda")
        kept = []
        for i in range(0, 4 * self.depth, 4):
            h, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
            ra.ra_layernorm_forward(x, w[i], w[i + 1], h, mean, rstd)
            a = torch.relu(h @ w[i + 2].t())
            kept.append((x, h, mean, rstd, a))
            x = x + a @ w[i + 3].t()
        i = 4 * self.depth
        h, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        ra.ra_layernorm_forward(x, w[i], w[i + 1], h, mean, rstd)
        error = (h @ w[i + 2].t()).float() - target
        dy = (error * (2.0 / error.numel())).to(BF16)
        g[i + 2].copy_(dy.t() @ h)
        dx = torch.empty_like(x)
        ra.ra_layernorm_backward(dy @ w[i + 2], x, w[i], mean, rstd, dx, g[i], g[i + 1], workspace=scratch)
        for i in reversed(range(0, 4 * self.depth, 4)):
            x, h, mean, rstd, a = kept.pop()
            g[i + 3].copy_(dx.t() @ a)
            da = (dx @ w[i + 3]) * (a > 0)
            g[i + 2].copy_(da.t() @ h)
            through = torch.empty_like(x)
            ra.ra_layernorm_backward(da @ w[i + 2], x, w[i], mean, rstd, through, g[i], g[i + 1], workspace=scratch)
            dx = dx + through
        return error.square().mean()


class Trainer:
    def __init__(self, model: Model, ranks: int, moments: str, max_norm: float = 1.0, weight_decay: float = 0.01):
        self.model, self.max_norm, self.steps = model, max_norm, 0
        self.grads = [torch.empty(model.total, dtype=BF16, device="cuda") for _ in range(ranks)]
        self.buckets = ra.ra_bucket_plan(model.counts, 1 << 20, 2)
        self.norm = torch.zeros(2, device="cuda")  # the norm, and the factor that clips it
        self.workspace = torch.zeros(ra.ra_grad_norm_workspace(), dtype=torch.uint8, device="cuda")
        params, grads = model.cut(model.master), model.cut(self.grads[0])
        decay = [weight_decay if len(s) == 2 else 0.0 for s in model.shapes]
        if moments == "8bit":
            scales = [torch.zeros(-(-n // ra.RA_ADAMW_BLOCK), device="cuda") for n in model.counts]
            state = ([torch.zeros(n, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for n in model.counts],
                     [torch.zeros(n, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for n in model.counts],
                     scales, [s.clone() for s in scales])
        else:
            state = ([torch.zeros_like(p) for p in params], [torch.zeros_like(p) for p in params])
        self.list = ra.grad_tensors([self.grads[0]])
        self.tensors = ra.adamw_tensors(params, grads, *state, weight_decay=decay, copies=model.cut(model.weights))

    def step(self, batches, lr: float):
        """One step on one (x, target) pair per rank; the ranks' mean loss."""
        losses = [self.model.loss_and_gradients(x, y, g) for (x, y), g in zip(batches, self.grads)]
        ra.ra_allreduce_buckets(self.grads, self.grads, self.buckets, "avg")
        ra.ra_grad_norm(self.list, self.max_norm, self.norm, self.workspace)
        self.steps += 1
        ra.ra_adamw(self.tensors, lr=lr, step=self.steps, grad_scale=self.norm[1:], seed=1)
        return torch.stack(losses).mean()


def samples(width: int, outputs: int, rows: int, gen):
    """Inputs, and targets that a fixed non-linear map makes of them."""
    fixed = torch.Generator(device="cuda").manual_seed(1234)
    a = torch.randn(width, outputs, generator=fixed, device="cuda") * width ** -0.5
    x = torch.randn(rows, width, generator=gen, device="cuda")
    return x.to(BF16), torch.tanh(x.to(BF16).float() @ a)


def train(ranks=4, steps=30, moments="f32", width=512, depth=4, rows=1024, outputs=64, lr=2e-3, show=None):
    model = Model(width, depth, outputs, seed=0)
    trainer = Trainer(model, ranks, moments)
    gen = torch.Generator(device="cuda").manual_seed(7)
    losses = []
    for k in range(steps):
        loss = trainer.step([samples(width, outputs, rows, gen) for _ in range(ranks)], lr)
        losses.append(loss)
        if show and (k % 5 == 0 or k == steps - 1):
            show(f"step {k + 1:4d}  loss {float(loss):.5f}  gradient norm {float(trainer.norm[0]):.4f}")
    return [float(v) for v in losses]


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--ranks", type=int, default=4)
    p.add_argument("--steps", type=int, default=30)
    p.add_argument("--moments", choices=["f32", "8bit"], default="f32")
    p.add_argument("--width", type=int, default=512)
    p.add_argument("--depth", type=int, default=4)
    args = p.parse_args()
    train(args.ranks, args.steps, args.moments, args.width, args.depth, show=print)
