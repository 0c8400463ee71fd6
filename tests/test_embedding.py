"""ra_embedding_forward / ra_embedding_backward against the formulas in 64 bits.

Tolerances come from the arithmetic, before any run. With u = 2^-24 the scaled
value is off by u of itself and the sum with an accumulated one by u of the sum;
a sum of n fp32 terms in any order is off by at most n u sum|term|. A stored
result adds half a step of its type."""

import pytest
import torch

U = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
ROUND = {F32: U, F16: 2.0 ** -11, BF16: 2.0 ** -8}
STEP = {F32: 2.0 ** -149, F16: 2.0 ** -25, BF16: 2.0 ** -134}
I32, I64 = torch.int32, torch.int64


@pytest.fixture(scope="module")
def ra():
    from ring_all_reduce_02_gb300 import build, ra as binding

    build.build()
    return binding


def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def matrix(rows, cols, dtype, gen, std=1.0, pad=0, shift=0):
    """A [rows, cols] view with `pad` elements between rows, `shift` elements past an allocation's start."""
    stride = cols + pad
    base = torch.full((rows * stride + shift + 1,), 7.0, dtype=dtype, device="cuda")
    v = base[shift:].as_strided((rows, cols), (stride, 1))
    v.copy_(torch.randn(rows, cols, generator=gen, dtype=torch.float64) * std)
    return v


def draw_tokens(kind, rows, vocab, gen, dtype):
    if kind == "text":  # the k-th token about 1/k as often as the first
        t = (torch.rand(rows, generator=gen, dtype=torch.float64) * torch.tensor(float(vocab + 1)).log()).expm1().long()
    elif kind == "one":
        t = torch.full((rows,), vocab // 2)
    elif kind == "ends":
        t = torch.randint(0, 2, (rows,), generator=gen) * (vocab - 1)
    elif kind == "descending":
        t = vocab - 1 - torch.arange(rows) % vocab
    else:
        t = torch.randint(0, vocab, (rows,), generator=gen)
    return t.clamp(0, vocab - 1).to(dtype).cuda()


def assert_within(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = (got - want).abs() - tol
    assert (bad <= 0).all(), f"{what}: off by {float((got - want).abs().max())}, {float(bad.max())} over the bound"


def check_forward(ra, table, tokens, out, scale, accumulate):
    old = out.double().clone()
    want = table.double()[tokens.long()] * scale
    tol = 2 * U * want.abs()
    if accumulate:
        want = want + old
        tol = tol + U * want.abs()
    ra.ra_embedding_forward(table, tokens, out, scale=scale, accumulate=accumulate)
    assert_within(out, want, 1.01 * tol + ROUND[out.dtype] * want.abs() + STEP[out.dtype], "out")


def check_backward(ra, dy, tokens, dtable, scale, accumulate, padding=None, workspace=None):
    vocab, cols = dtable.shape
    rows = dy.shape[0]
    t = tokens.long()
    keep = (t >= 0) & (t < vocab)
    if padding is not None:
        keep &= t != padding
    terms = dy.double()[keep] * scale
    old = dtable.double().clone()
    zero = torch.zeros(vocab, cols, dtype=torch.float64, device="cuda")
    want, size = zero.index_add(0, t[keep], terms), zero.index_add(0, t[keep], terms.abs())
    counts = torch.zeros(vocab, dtype=torch.float64, device="cuda").index_add(0, t[keep], torch.ones(int(keep.sum()), dtype=torch.float64, device="cuda"))
    tol = (counts[:, None] + 2) * U * size
    if accumulate:
        want = want + old
        tol = tol + U * want.abs()
    if workspace is None:
        workspace = torch.full((ra.ra_embedding_workspace(rows, cols, vocab),), 255, dtype=torch.uint8, device="cuda")
    ra.ra_embedding_backward(dy, tokens, dtable, scale=scale, accumulate=accumulate, padding=padding, workspace=workspace)
    assert_within(dtable, want, 1.01 * tol + ROUND[dtable.dtype] * want.abs() + STEP[dtable.dtype], "dtable")
    if accumulate:
        untouched = counts == 0
        assert torch.equal(dtable.double()[untouched], old[untouched])


SHAPES = [(1, 1, 1), (1, 1024, 50), (2, 3, 2), (5, 31, 7), (33, 64, 100), (64, 33, 3), (100, 100, 1000), (255, 72, 40), (256, 264, 30), (257, 128, 64),
          (1000, 72, 5000), (1025, 257, 300), (3000, 8, 40), (4099, 96, 700), (9001, 40, 50257), (20000, 16, 11)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,index", [(BF16, I64), (F16, I32), (F32, I64)])
@pytest.mark.parametrize("rows,cols,vocab", SHAPES)
def test_forward_and_backward(ra, rows, cols, vocab, dtype, index):
    gpu()
    for accumulate in (False, True):
        for kind in ("text", "any"):
            gen = torch.Generator().manual_seed(rows * 1009 + cols)
            tokens = draw_tokens(kind, rows, vocab, gen, index)
            check_forward(ra, matrix(vocab, cols, dtype, gen), tokens, matrix(rows, cols, dtype, gen), 5.5, accumulate)
            check_backward(ra, matrix(rows, cols, dtype, gen), tokens, matrix(vocab, cols, dtype, gen), 0.3, accumulate)


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [300, 2 ** 17 - 1, 2 ** 17])
@pytest.mark.parametrize("rows", [2048, 2049, 4096, 4097, 8192, 8193, 16384, 16385, 24576, 24577, 32768, 32769])
def test_ends_of_the_sorts_ranges(ra, rows, vocab):
    gpu()
    gen = torch.Generator().manual_seed(rows + vocab)
    for kind in ("any", "descending"):
        tokens = draw_tokens(kind, rows, vocab, gen, I64)
        tokens[::97] = vocab - 1
        check_backward(ra, matrix(rows, 8, BF16, gen), tokens, matrix(vocab, 8, F32, gen), 1.0, True, padding=7)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["one", "ends", "descending"])
@pytest.mark.parametrize("rows,cols,vocab", [(1, 64, 9), (31, 40, 1), (256, 72, 3), (300, 65, 2), (5000, 64, 333), (40000, 24, 50257), (70001, 17, 9)])
def test_orders_and_repeats(ra, rows, cols, vocab, kind):
    gpu()
    gen = torch.Generator().manual_seed(rows + cols)
    tokens = draw_tokens(kind, rows, vocab, gen, I64)
    for accumulate in (False, True):
        check_backward(ra, matrix(rows, cols, BF16, gen), tokens, matrix(vocab, cols, BF16, gen), 1.0, accumulate)
        check_backward(ra, matrix(rows, cols, BF16, gen), tokens, matrix(vocab, cols, F32, gen), 1.0, accumulate)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("cols,pad,shift", [(64, 8, 0), (256, 3, 0), (1024, 1, 1), (1024, 0, 1), (1000, 24, 4), (96, 16, 8), (515, 2, 3)])
def test_strides_and_alignment(ra, dtype, cols, pad, shift):
    gpu()
    gen = torch.Generator().manual_seed(cols + 31 * pad + shift)
    rows, vocab = 200, 90
    tokens = draw_tokens("any", rows, vocab, gen, I32)
    for other in (0, shift):
        table, out = matrix(vocab, cols, dtype, gen, pad=pad, shift=shift), matrix(rows, cols, dtype, gen, pad=pad, shift=other)
        check_forward(ra, table, tokens, out, 2.0, True)
        dy, dtable = matrix(rows, cols, dtype, gen, pad=pad, shift=other), matrix(vocab, cols, dtype, gen, pad=pad, shift=shift)
        check_backward(ra, dy, tokens, dtable, 2.0, False)
        check_backward(ra, dy, tokens, dtable, 2.0, True)
    if pad:  # what lies between the rows stays
        flat = dtable.as_strided((vocab * (cols + pad),), (1,)).view(vocab, cols + pad)
        assert (flat[:-1, cols:] == 7).all()


@pytest.mark.gpu
def test_tokens_outside_the_vocabulary_and_padding(ra):
    gpu()
    gen = torch.Generator().manual_seed(3)
    rows, cols, vocab = 500, 72, 60
    for index in (I32, I64):
        tokens = draw_tokens("any", rows, vocab, gen, index)
        tokens[::7] = 5
        bad = [0, 3, 250, 499]
        for i, v in zip(bad, (-1, vocab, -2 ** 31, 2 ** 31 - 1) if index is I32 else (-1, vocab, 2 ** 40 + 1, -2 ** 63)):
            tokens[i] = v
        table, out = matrix(vocab, cols, F32, gen), matrix(rows, cols, F32, gen)
        ra.ra_embedding_forward(table, tokens, out)
        good = torch.ones(rows, dtype=torch.bool, device="cuda")
        good[bad] = False
        assert torch.isnan(out[~good]).all() and torch.equal(out[good], table[tokens.long()[good]])
        dy = matrix(rows, cols, F32, gen)
        dy[bad] = float("nan")  # what does not count is not added, whatever it holds
        for padding in (5, None, vocab, -7):
            for accumulate in (False, True):
                check_backward(ra, dy, tokens, matrix(vocab, cols, F32, gen), 1.0, accumulate, padding=padding)
        dy[tokens == 5] = float("inf")
        check_backward(ra, dy, tokens, matrix(vocab, cols, F32, gen), 1.0, False, padding=5)


@pytest.mark.gpu
def test_infinities_and_nan_reach_their_token_alone(ra):
    gpu()
    gen = torch.Generator().manual_seed(4)
    rows, cols, vocab = 3000, 40, 100
    tokens = draw_tokens("any", rows, vocab, gen, I64)
    tokens[100], tokens[2000] = 11, 13
    dy = matrix(rows, cols, BF16, gen)
    dy[100, 3], dy[2000, 4] = float("inf"), float("nan")
    dtable = torch.empty(vocab, cols, dtype=BF16, device="cuda")
    ws = torch.empty(ra.ra_embedding_workspace(rows, cols, vocab), dtype=torch.uint8, device="cuda")
    ra.ra_embedding_backward(dy, tokens, dtable, workspace=ws)
    assert dtable[11, 3] == float("inf") and torch.isnan(dtable[13, 4])
    dtable[11, 3] = dtable[13, 4] = 0
    assert torch.isfinite(dtable).all()


@pytest.mark.gpu
def test_no_rows(ra):
    gpu()
    none, tokens = torch.empty(0, 16, device="cuda"), torch.empty(0, dtype=I64, device="cuda")
    table = torch.ones(9, 16, device="cuda")
    ws = torch.empty(max(16, ra.ra_embedding_workspace(0, 16, 9)), dtype=torch.uint8, device="cuda")
    ra.ra_embedding_forward(table, tokens, none)
    ra.ra_embedding_backward(none, tokens, table, accumulate=True, workspace=ws)
    assert (table == 1).all()
    ra.ra_embedding_backward(none, tokens, table, workspace=ws)
    assert (table == 0).all()


@pytest.mark.gpu
def test_same_bits_again_on_another_stream_and_in_a_graph(ra):
    gpu()
    gen = torch.Generator().manual_seed(6)
    rows, cols, vocab = 9000, 136, 2000
    tokens = draw_tokens("text", rows, vocab, gen, I64)
    dy, table = matrix(rows, cols, F32, gen), matrix(vocab, cols, F32, gen)
    ws = torch.empty(ra.ra_embedding_workspace(rows, cols, vocab), dtype=torch.uint8, device="cuda")

    def both(o, stream=None):
        ra.ra_embedding_forward(table, tokens, o[0], scale=3.0, stream=stream)
        ra.ra_embedding_backward(dy, tokens, o[1], scale=3.0, workspace=ws, stream=stream)
        ra.ra_embedding_backward(dy, tokens, o[2], scale=3.0, accumulate=True, workspace=ws, stream=stream)

    def outputs():
        return [torch.zeros_like(dy), torch.zeros_like(table), torch.ones_like(table)]

    want = outputs()
    both(want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = outputs()
        torch.cuda.synchronize()
        both(got, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = outputs()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        both(got)
    torch.cuda.synchronize()
    assert (got[0] == 0).all()
    for _ in range(2):
        got[2].fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_more_than_32_bits_of_elements(ra):
    # tables and rows of 2.2e9 elements: the first and the last tokens
    gpu()
    cols = 8192
    vocab = rows = (1 << 31) // cols + 301
    gen = torch.Generator().manual_seed(8)
    table = torch.zeros(vocab, cols, dtype=BF16, device="cuda")
    table[-1], table[0] = torch.randn(cols, generator=gen).to(BF16).cuda(), torch.randn(cols, generator=gen).to(BF16).cuda()
    tokens = torch.randint(1, vocab - 1, (rows,), generator=gen).cuda()
    tokens[0], tokens[-1], tokens[-2] = vocab - 1, 0, vocab - 1
    out = torch.empty(rows, cols, dtype=BF16, device="cuda")
    ra.ra_embedding_forward(table, tokens, out)
    assert torch.equal(out[0], table[-1]) and torch.equal(out[-1], table[0]) and torch.equal(out[-2], table[-1])
    assert (out[1:-2] == 0).all()
    ws = torch.empty(ra.ra_embedding_workspace(rows, cols, vocab), dtype=torch.uint8, device="cuda")
    ra.ra_embedding_backward(out, tokens, table.fill_(7), workspace=ws)
    assert torch.equal(table[0], out[-1]) and torch.equal(table[-1].float(), (out[0].float() * 2))
    assert (table[1:-1] == 0).all()


# Fake addresses that are never dereferenced: every case is refused on the host.
BASE = 0x7F0000000000
MB = 1 << 20


def test_forward_refusals(ra):
    def call(table=BASE, ts=64, tokens=BASE + 4 * MB, size=8, out=BASE + 8 * MB, os=64, acc=0, rows=16, cols=64, vocab=100, scale=1.0, dt=2):
        return ra.lib().ra_embedding_forward(table, ts, tokens, size, out, os, acc, rows, cols, vocab, scale, dt, None)

    bad, alias = ra.RA_ERR_INVALID_ARG, ra.RA_ERR_ALIAS
    assert call(dt=3) == ra.RA_ERR_UNSUPPORTED and call(dt=9) == bad
    assert call(size=2) == call(size=0) == call(ts=63) == call(os=63) == bad
    assert call(table=0) == call(tokens=0) == call(out=0) == bad
    assert call(table=BASE + 1) == call(tokens=BASE + 4 * MB + 4) == call(out=BASE + 8 * MB + 1) == bad
    assert call(scale=float("inf")) == call(scale=float("nan")) == call(scale=1e39) == call(scale=-1e39) == bad
    assert call(rows=1 << 31) == call(vocab=1 << 31) == call(cols=1 << 57, ts=1 << 57, os=1 << 57) == bad
    assert call(out=BASE + 2) == call(out=BASE, os=65) == call(out=BASE + 4 * MB) == alias
    assert call(rows=0) == call(cols=0, ts=0, os=0) == ra.RA_SUCCESS


def test_backward_refusals(ra):
    need = ra.ra_embedding_workspace(16, 64, 100)

    def call(dy=BASE, ds=64, tokens=BASE + 4 * MB, size=8, pad=-1, dt=BASE + 8 * MB, ts=64, acc=0, rows=16, cols=64, vocab=100, scale=1.0,
             dtype=2, tdtype=2, ws=BASE + 16 * MB, nws=need):
        return ra.lib().ra_embedding_backward(dy, ds, tokens, size, pad, dt, ts, acc, rows, cols, vocab, scale, dtype, tdtype, ws, nws, None)

    bad, alias = ra.RA_ERR_INVALID_ARG, ra.RA_ERR_ALIAS
    assert need > 0 and ra.ra_embedding_workspace(1 << 31, 1, 1) == ra.ra_embedding_workspace(1, 1, 1 << 31) == 0
    assert call(dtype=3) == call(dtype=2, tdtype=1) == call(dtype=0, tdtype=2) == ra.RA_ERR_UNSUPPORTED
    assert call(dtype=5) == call(tdtype=-1) == bad
    assert call(size=3) == call(ds=63) == call(ts=63) == call(scale=float("nan")) == call(scale=-1e39) == bad
    assert call(dy=0) == call(tokens=0) == call(dt=0) == call(ws=0) == call(nws=need - 1) == call(ws=BASE + 16 * MB + 8) == bad
    assert call(rows=1 << 31) == call(vocab=1 << 31) == bad
    assert call(dt=BASE + 2) == call(dt=BASE, ts=65) == call(ws=BASE) == call(ws=BASE + 8 * MB) == call(dt=BASE + 4 * MB) == alias
    assert call(rows=0, acc=1) == call(cols=0, ds=0, ts=0) == call(vocab=0) == ra.RA_SUCCESS


def test_binding_refusals(ra):
    x, t = torch.zeros(4, 8), torch.zeros(4, dtype=I64)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_embedding_forward(x, t, x)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_embedding_backward(x, t, x, workspace=x)
    with pytest.raises(ValueError, match="two dimensions"):
        ra.ra_embedding_forward(x[0], t, x)
    with pytest.raises(TypeError):
        ra.ra_embedding_forward(x.int(), t, x)
