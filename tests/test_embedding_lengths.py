"""ra_embedding_backward at the ends of its lengths: no rows at all, into tables of either sort, and more tokens than a
pass of the sort has CTAs for."""

import pytest
import torch

from test_embedding import BF16, F16, F32, I64, check_backward, gpu, matrix, ra  # noqa: F401


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,tdtype", [(BF16, BF16), (BF16, F32), (F16, F16), (F32, F32)])
@pytest.mark.parametrize("vocab", [1, 9, 2 ** 17 - 1, 2 ** 17, 200_003])
def test_no_rows(ra, vocab, dtype, tdtype):  # noqa: F811
    # a rank without tokens: the whole table is zero, and with accumulate what it was; the columns beside it stay
    gpu()
    cols, pad = 24, 8
    none, tokens = torch.empty(0, cols, dtype=dtype, device="cuda"), torch.empty(0, dtype=I64, device="cuda")
    for width in (cols, cols + pad):
        wide = torch.full((vocab, width), 7.0, dtype=tdtype, device="cuda")
        ws = torch.full((ra.ra_embedding_workspace(0, cols, vocab),), 255, dtype=torch.uint8, device="cuda")
        ra.ra_embedding_backward(none, tokens, wide[:, :cols], accumulate=True, workspace=ws)
        assert (wide == 7).all()
        ra.ra_embedding_backward(none, tokens, wide[:, :cols], workspace=ws)
        assert (wide[:, :cols] == 0).all() and (wide[:, cols:] == 7).all()
