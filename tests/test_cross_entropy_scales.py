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


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,cols,vocab", [(130, 64, 400), (700, 129, 3000)])
def test_rows_of_very_different_dloss(ra, dtype, rows, cols, vocab):  # noqa: F811
    # g has one scale for all rows: each row is held to what that leaves it. fp16 has its 11 bits of a g down to 2^-28 of the
    # largest |dloss|, and multiples of 2^-38 of it below; bf16 has its 8 bits of every one
    gpu()
    gen = generator(31)
    h, w = matrix(rows, cols, dtype, gen), matrix(vocab, cols, dtype, gen, std=0.02)
    targets = draw_targets(rows, vocab, gen)
    lse = check_forward(ra, h, w, targets)
    powers = torch.randint(-24, 1, (rows,), generator=gen, device="cuda")
    powers[7] = 0
    dloss = 2.0 ** 16 * torch.ldexp(torch.rand(rows, generator=gen, device="cuda") + 0.5, powers)
    check_backward(ra, h, w, targets, lse, dloss, torch.empty_like(h), torch.empty_like(w, dtype=F32))
    # a row alone has a scale of its own
    for i in (0, rows - 1):
        check_backward(ra, h[i:i + 1], w, targets[i:i + 1], lse[i:i + 1].contiguous(), dloss[i:i + 1].contiguous(), torch.empty_like(h[i:i + 1]),
                       torch.empty_like(w, dtype=F32))
