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


def whole_numbers(rows, cols, gen):
    """dy of small whole numbers: their sums are exact in fp32, in any order."""
    return torch.randint(-2, 3, (rows, cols), generator=gen, device="cuda").to(BF16)


def exact_gradient(dy, tokens, vocab):
    """In 64-bit sums, by parts: whole numbers."""
    want = torch.zeros(vocab, dy.shape[1], dtype=torch.float64, device="cuda")
    for a in range(0, len(tokens), 1 << 20):
        want.index_add_(0, tokens[a:a + (1 << 20)], dy[a:a + (1 << 20)].double())
    return want


def check_exactly(ra, dy, tokens, vocab):  # noqa: F811
    want = exact_gradient(dy, tokens, vocab)
    assert float(want.abs().max()) < 2 ** 24
    ws = torch.full((ra.ra_embedding_workspace(len(tokens), dy.shape[1], vocab),), 255, dtype=torch.uint8, device="cuda")
    dtable = torch.full((vocab, dy.shape[1]), 7.0, device="cuda")
    ra.ra_embedding_backward(dy, tokens, dtable, workspace=ws)
    assert torch.equal(dtable.double(), want)
    ra.ra_embedding_backward(dy, tokens, dtable, accumulate=True, workspace=ws)
    assert torch.equal(dtable.double(), 2 * want)


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [40, 200_003])
@pytest.mark.parametrize("cols", [8, 3])
def test_tokens_over_many_spans(ra, vocab, cols):  # noqa: F811
    # a CTA finds where a token that reaches over it starts and ends, 1 to 2000 CTAs away, at and beside powers of 32
    gpu()
    gen = torch.Generator(device="cuda").manual_seed(vocab + cols)
    spans = [1, 2, 31, 32, 33, 34, 63, 64, 65, 100, 1023, 1024, 1025, 1056, 1057, 1500]
    for first in (0, 1, 255):  # places before the first of them
        lengths = torch.tensor([first] + [n * 256 + d for n, d in zip(spans, (0, 1, -1, 128) * 4)])
        runs = torch.repeat_interleave(torch.arange(len(lengths)), lengths).cuda()
        tokens = runs[torch.randperm(len(runs), generator=gen, device="cuda")] * (vocab // 40)
        check_exactly(ra, whole_numbers(len(tokens), cols, gen), tokens, vocab)


def fastest(call, times=5):
    best = float("inf")
    for k in range(times + 1):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        call()
        end.record()
        torch.cuda.synchronize()
        best = min(best, start.elapsed_time(end)) if k else best
    return best


@pytest.mark.gpu
def test_one_tokens_time_grows_with_its_places(ra):  # noqa: F811
    # 8 times the places in at most 14 times the time. A search from CTA to CTA would take 19 times it: the ends are as many
    # CTAs away as there are
    gpu()
    cols, vocab, times = 64, 50257, []
    for rows in (1 << 20, 1 << 23):
        dy, tokens = torch.ones(rows, cols, dtype=BF16, device="cuda"), torch.full((rows,), 77, dtype=I64, device="cuda")
        dtable = torch.empty(vocab, cols, device="cuda")
        ws = torch.empty(ra.ra_embedding_workspace(rows, cols, vocab), dtype=torch.uint8, device="cuda")
        times.append(fastest(lambda: ra.ra_embedding_backward(dy, tokens, dtable, workspace=ws)))
        assert (dtable[77] == rows).all() and float(dtable.sum()) == rows * cols
    assert times[1] <= 14 * times[0], times


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [40, 50257, 200_003])
@pytest.mark.parametrize("rows", [304 * 4096 - 1, 304 * 4096, 304 * 4096 + 1, 2 * 304 * 4096 + 1, 10_100_003])
def test_more_tiles_than_a_pass_has_ctas(ra, rows, vocab):  # noqa: F811
    gpu()
    gen = torch.Generator(device="cuda").manual_seed(rows + vocab)
    u = torch.rand(rows, generator=gen, device="cuda", dtype=torch.float64)
    check_exactly(ra, whole_numbers(rows, 5, gen), (u * u * vocab).long(), vocab)


@pytest.mark.gpu
def test_the_sorts_time_grows_with_the_tokens(ra):  # noqa: F811
    # 8 times the tokens in at most 12 times the time. Were each tile a CTA's, which reads the counts of all, it would be 18 times
    gpu()
    cols, vocab, times = 8, 50257, []
    gen = torch.Generator(device="cuda").manual_seed(1)
    for rows in (1 << 22, 1 << 25):
        dy, tokens = torch.ones(rows, cols, dtype=BF16, device="cuda"), torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
        dtable = torch.empty(vocab, cols, device="cuda")
        ws = torch.empty(ra.ra_embedding_workspace(rows, cols, vocab), dtype=torch.uint8, device="cuda")
        times.append(fastest(lambda: ra.ra_embedding_backward(dy, tokens, dtable, workspace=ws)))
        assert torch.equal(dtable[:, 0].long(), torch.bincount(tokens, minlength=vocab))
    assert times[1] <= 12 * times[0], times
