"""Rows without a loss: whatever their hidden states, dloss and lse hold, every result has the bits that it has with zeros
there."""

import pytest
import torch

from test_cross_entropy import BF16, F16, F32, I32, draw_targets, generator, gpu, matrix, ra, scratch  # noqa: F401

PATTERNS = {"all but the first": lambda i, n: i > 0, "all but the last": lambda i, n: i < n - 1, "every third": lambda i, n: i % 3 == 0,
            "first half": lambda i, n: i < n // 2, "blocks": lambda i, n: i // 64 % 2 == 1, "all": lambda i, n: True}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("rows,cols,shift", [(50, 64, 0), (700, 136, 0), (513, 77, 1), (2500, 40, 0)])
def test_ignored_rows_change_no_bit(ra, rows, cols, shift, pattern, dtype):  # noqa: F811
    gpu()
    vocab = 1500
    gen = generator(rows + cols)
    ignored = torch.tensor([PATTERNS[pattern](i, rows) for i in range(rows)], device="cuda")
    h, w = matrix(rows, cols, dtype, gen, shift=shift), matrix(vocab, cols, dtype, gen, std=0.2, shift=shift)
    targets = draw_targets(rows, vocab, gen, I32)
    targets[ignored] = -100
    dloss = torch.randn(rows, generator=gen, device="cuda")
    anything = torch.tensor([float("nan"), float("inf"), float("-inf"), 3e38 if dtype is BF16 else 6e4], device="cuda")
    anything = anything[torch.arange(rows, device="cuda") % 4][ignored]

    def results(fill):
        h[ignored] = fill[:, None].to(dtype)
        dloss[ignored] = fill
        loss, lse, dh = torch.full((rows,), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda"), torch.full_like(h, 7.0)
        ra.ra_cross_entropy_forward(h, w, targets, loss, lse, workspace=scratch(ra, h, w))
        out = [loss, lse.clone(), dh]
        lse[ignored] = fill
        for dw in (torch.full_like(w, 7.0), torch.full((vocab, cols), 7.0, dtype=F32, device="cuda")):
            for accumulate in (False, True):
                ra.ra_cross_entropy_backward(h, w, targets, lse, dloss, dh, dw, accumulate=accumulate, workspace=scratch(ra, h, w, backward=True))
            out.append(dw)
        return out

    clean, poisoned = results(torch.zeros_like(anything)), results(anything)
    for a, b in zip(clean, poisoned):
        assert torch.isfinite(a).all() and torch.equal(a, b)
    assert (clean[0][ignored] == 0).all() and (clean[1][ignored] == 0).all() and (clean[2][ignored] == 0).all()
    if pattern == "all":
        assert all((dw == 0).all() for dw in clean[3:])
