"""The cross entropy's gradients for dloss of extreme and of very different sizes."""

import pytest
import torch

from test_cross_entropy import BF16, F16, F32, check_backward, check_forward, draw_targets, generator, gpu, matrix, ra  # noqa: F401


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("size", [1e-34, 1e-36, 1e-38, 1e-40, 1e36])
@pytest.mark.parametrize("cols,shift", [(64, 0), (65, 1)])
def test_extreme_dloss(ra, dtype, size, cols, shift):  # noqa: F811
    # the factor that takes g's scale back is a normal number, or the gradient loses bits that fp32 has: with fp16's
    # factor of 2^-14 a scale below 2^-112 would make it subnormal. 1e-40 is a subnormal dloss itself
    gpu()
    rows, vocab = 130, 400
    gen = generator(21)
    h, w = matrix(rows, cols, dtype, gen, std=8.0, shift=shift), matrix(vocab, cols, dtype, gen, std=0.02, shift=shift)
    targets = draw_targets(rows, vocab, gen)
    lse = check_forward(ra, h, w, targets)
    dloss = torch.randn(rows, generator=gen, device="cuda").clamp(-3, 3) * size
    for accumulate in (False, True):
        dw = torch.zeros(vocab, cols, dtype=F32, device="cuda")
        check_backward(ra, h, w, targets, lse, dloss, torch.empty_like(h) if dtype is BF16 else None, dw, accumulate)
