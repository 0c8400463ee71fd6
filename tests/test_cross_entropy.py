"""ra_cross_entropy_forward / ra_cross_entropy_backward against the formulas in 64 bits.

Tolerances come from the arithmetic, before any run. With u = 2^-24: products of
16-bit values are exact in fp32; a sum of n of them in any order, each addition
cut off rather than rounded, is off by at most 2 n u sum|term|. An exponential is
off by its argument's rounding (3 u of the argument's size) and 4 u of itself.
g is rounded once more by half a step of the operands' type."""

import pytest
import torch

U = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
ROUND = {F32: U, F16: 2.0 ** -11, BF16: 2.0 ** -8}
STEP = {F32: 2.0 ** -149, F16: 2.0 ** -25, BF16: 2.0 ** -134}
I32, I64 = torch.int32, torch.int64
IGNORE = -100


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
    v.copy_(torch.randn(rows, cols, generator=gen, device="cuda") * std)
    return v


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def draw_targets(rows, vocab, gen, index=I64, ignored=()):
    t = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    t[list(ignored)] = IGNORE
    return t.to(index)


def scratch(ra, h, w, backward=False):
    # its contents do not matter: bytes of 255 are NaN
    # and where it starts (on a 16-byte boundary) does not either
    return torch.full((16 + ra.ra_cross_entropy_workspace(h, w, backward=backward),), 255, dtype=torch.uint8, device="cuda")[16:]


def assert_within(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = (got - want).abs() - tol
    assert (bad <= 0).all(), f"{what}: off by {float((got - want).abs().max())}, {float(bad.max())} over the bound"


def definition(h, w, targets):
    """Counted rows, their logits, how far those may be off, lse, and how far that may be off."""
    counts = targets != IGNORE
    h64, w64 = h.double()[counts], w.double()
    logits = h64 @ w64.t()
    off = 2 * (w.shape[1] + 16) * U * (h64.abs() @ w64.abs().t())
    lse = torch.logsumexp(logits, 1)
    p = torch.exp(logits - lse[:, None])
    lse_off = (p * (off + 3 * U * (logits - logits.amax(1, keepdim=True)).abs())).sum(1) + (400 + w.shape[0] / 4096) * U + 2 * U * lse.abs()
    return counts, h64, w64, logits, off, lse, lse_off


def check_forward(ra, h, w, targets, loss=None, lse=None):
    rows = h.shape[0]
    loss = torch.full((rows,), 7.0, device="cuda") if loss is None else loss
    lse = torch.full((rows,), 7.0, device="cuda") if lse is None else lse
    ra.ra_cross_entropy_forward(h, w, targets, loss, lse, ignore=IGNORE, workspace=scratch(ra, h, w))
    counts, _, _, logits, off, want, want_off = definition(h, w, targets)
    assert (loss[~counts] == 0).all() and (lse[~counts] == 0).all()
    at = targets[counts].long()[:, None]
    assert_within(lse[counts], want, want_off, "lse")
    assert_within(loss[counts], want - logits.gather(1, at)[:, 0], want_off + off.gather(1, at)[:, 0] + 2 * U * want.abs(), "loss")
    return lse


def check_backward(ra, h, w, targets, lse, dloss, dh, dw, accumulate=False):
    counts, h64, w64, logits, off, _, _ = definition(h, w, targets)
    at = targets[counts].long()
    lse64 = lse.double()[counts][:, None]
    d = torch.ones(len(at), dtype=torch.float64, device="cuda") if dloss is None else dloss.double()[counts]
    p = torch.exp(logits - lse64)
    p_off = p * (off + 3 * U * (logits - lse64).abs() + 8 * U)
    g = p.clone()
    g[torch.arange(len(at), device="cuda"), at] -= 1
    largest = d.abs().max() if len(d) else 0.0
    # the subtraction, the product, the division; the rounding to the operands' type (fp16: its smallest step is
    # 2^-24 where the largest |dloss| is 2^14)
    g_off = (p_off + 4 * U * g.abs()) * d.abs()[:, None]
    g = g * d[:, None]
    g_off = g_off + ROUND[h.dtype] * 1.01 * g.abs() + largest * (2.0 ** -39 if h.dtype is F16 else 2.0 ** -120)
    old = None if dw is None else dw.double().clone()
    ra.ra_cross_entropy_backward(h, w, targets, lse, dloss, dh, dw, ignore=IGNORE, accumulate=accumulate,
                                 workspace=scratch(ra, h, w, backward=True))
    if dh is not None:
        want = g @ w64
        tol = (g_off + 2 * (w.shape[0] + 32) * U * g.abs()) @ w64.abs() * 1.01
        assert (dh[~counts] == 0).all()
        assert_within(dh[counts], want, tol + ROUND[dh.dtype] * want.abs() + STEP[dh.dtype], "dhidden")
    if dw is not None:
        want = g.t() @ h64
        tol = (g_off + 2 * (len(at) + 32) * U * g.abs()).t() @ h64.abs() * 1.01
        if accumulate:
            want = want + old
            tol = tol + 2 * U * want.abs()
        assert_within(dw, want, tol + ROUND[dw.dtype] * want.abs() + STEP[dw.dtype], "dweight")


def check_both(ra, h, w, targets, dloss, wdtype=None, accumulate=False, gen=None):
    lse = check_forward(ra, h, w, targets)
    dw = matrix(w.shape[0], w.shape[1], wdtype or w.dtype, gen or generator(1), std=0.1)
    check_backward(ra, h, w, targets, lse, dloss, torch.full_like(h, 7.0), dw, accumulate)


SHAPES = [(1, 1, 1), (1, 64, 2), (1, 1024, 5000), (2, 8, 255), (3, 7, 31), (31, 65, 256), (64, 128, 257), (127, 100, 1000), (128, 64, 512),
          (129, 63, 513), (255, 192, 300), (256, 256, 768), (257, 40, 2049), (300, 771, 1003), (513, 129, 700), (1000, 72, 5003),
          (61, 1024, 10007)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,cols,vocab", SHAPES)
def test_forward_and_backward(ra, rows, cols, vocab, dtype):
    gpu()
    gen = generator(rows * 1009 + cols * 31 + vocab)
    h, w = matrix(rows, cols, dtype, gen), matrix(vocab, cols, dtype, gen, std=2.0 / cols ** 0.5)
    dloss = torch.randn(rows, generator=gen, device="cuda") / rows
    check_both(ra, h, w, draw_targets(rows, vocab, gen, I64), dloss)
    check_both(ra, h, w, draw_targets(rows, vocab, gen, I32), None, wdtype=F32, accumulate=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("pattern", ["all", "all but the first", "all but the last", "every third", "first half", "blocks"])
def test_ignored_rows_hold_anything(ra, dtype, pattern):
    gpu()
    rows, cols, vocab = 700, 136, 1500
    gen = generator(5)
    ignored = {"all": range(rows), "all but the first": range(1, rows), "all but the last": range(rows - 1), "every third": range(0, rows, 3),
               "first half": range(rows // 2), "blocks": [i for i in range(rows) if i // 100 % 2]}[pattern]
    h, w = matrix(rows, cols, dtype, gen), matrix(vocab, cols, dtype, gen, std=0.2)
    targets = draw_targets(rows, vocab, gen, I64, ignored)
    dloss = torch.randn(rows, generator=gen, device="cuda")
    for i, v in zip(ignored, (float("nan"), float("inf"), float("-inf"))):
        h[i] = v
        dloss[i] = v
    lse = check_forward(ra, h, w, targets)
    lse[list(ignored)] = float("nan")  # not read
    clean = torch.where((targets != IGNORE)[:, None], h, torch.zeros_like(h))
    del clean
    check_backward(ra, h, w, targets, lse, dloss, torch.full_like(h, 7.0), matrix(vocab, cols, dtype, gen))


@pytest.mark.gpu
@pytest.mark.parametrize("ignore", [0, 3, -1, 2 ** 31 - 1])
def test_ignore_may_be_any_number(ra, ignore):
    gpu()
    rows, cols, vocab = 90, 64, 50
    gen = generator(6)
    h, w = matrix(rows, cols, BF16, gen), matrix(vocab, cols, BF16, gen)
    t = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    t[::4] = ignore
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    for index in (I32, I64):
        ra.ra_cross_entropy_forward(h, w, t.to(index), loss, lse, ignore=ignore, workspace=scratch(ra, h, w))
        same = torch.where(t == ignore, torch.full_like(t, IGNORE), t)
        want = check_forward(ra, h, w, same)
        assert torch.equal(lse, want) and ((loss == 0) == (t == ignore)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("cols,pad,shift", [(64, 8, 0), (64, 8, 8), (96, 3, 0), (128, 0, 1), (100, 4, 0), (200, 8, 4), (77, 1, 2)])
def test_strides_and_alignment(ra, dtype, cols, pad, shift):
    gpu()
    rows, vocab = 150, 600
    gen = generator(cols + pad)
    for other in (0, shift):
        h, w = matrix(rows, cols, dtype, gen, pad=pad, shift=other), matrix(vocab, cols, dtype, gen, std=0.1, pad=pad, shift=shift)
        targets = draw_targets(rows, vocab, gen)
        lse = check_forward(ra, h, w, targets)
        dh, dw = matrix(rows, cols, dtype, gen, pad=pad, shift=shift), matrix(vocab, cols, dtype, gen, pad=pad, shift=other)
        check_backward(ra, h, w, targets, lse, None, dh, dw, accumulate=True)
        if pad:  # what lies between the rows stays
            for m in (dh, dw):
                flat = m.as_strided((m.shape[0] * (cols + pad),), (1,)).view(m.shape[0], cols + pad)
                assert (flat[:-1, cols:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rows,cols,pad,vocab", [(70, 64, 64, 300), (70, 72, 8, 33), (300, 200, 56, 601), (9, 264, 248, 1025), (300, 65, 1, 290),
                                                 (40, 8, 8, 31)])
def test_columns_between_others(ra, dtype, accumulate, rows, cols, pad, vocab):
    # the gradients of a slice of a wider matrix's columns, of both types: its other columns and the rows behind it stay
    gpu()
    gen = generator(rows + cols)
    h, w = matrix(rows, cols, dtype, gen), matrix(vocab, cols, dtype, gen, std=0.1)
    targets = draw_targets(rows, vocab, gen, I64, [1])
    lse = check_forward(ra, h, w, targets)
    for wdtype in (dtype, F32):
        for first in (0, pad):
            wide = torch.full((vocab + 2, cols + pad), 7.0, dtype=wdtype, device="cuda")
            check_backward(ra, h, w, targets, lse, None, torch.full_like(h, 7.0), wide[:vocab, first:first + cols], accumulate)
            assert (wide[vocab:] == 7).all() and (wide[:, :first] == 7).all() and (wide[:, first + cols:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_one_gradient_alone(ra, dtype):
    gpu()
    rows, cols, vocab = 300, 96, 900
    gen = generator(9)
    h, w = matrix(rows, cols, dtype, gen), matrix(vocab, cols, dtype, gen, std=0.1)
    targets = draw_targets(rows, vocab, gen)
    lse = check_forward(ra, h, w, targets)
    check_backward(ra, h, w, targets, lse, None, torch.empty_like(h), None)
    check_backward(ra, h, w, targets, lse, None, None, torch.empty_like(w))
    check_backward(ra, h, w, targets, lse, None, None, torch.empty_like(w, dtype=F32))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("size", [0.0, 1e-30, 1e-6, 1e6, 1e30])
def test_gradients_of_any_size(ra, dtype, size):
    # g is held relative to the largest |dloss|: no dloss underflows or overflows fp16
    gpu()
    rows, cols, vocab = 130, 64, 400
    gen = generator(10)
    h, w = matrix(rows, cols, dtype, gen), matrix(vocab, cols, dtype, gen, std=0.3)
    targets = draw_targets(rows, vocab, gen)
    lse = check_forward(ra, h, w, targets)
    dloss = torch.randn(rows, generator=gen, device="cuda") * size
    dloss[::5] = 0
    wide = 1e-30 <= size <= 1e30 and dtype is BF16 or size in (0.0, 1e-6)
    check_backward(ra, h, w, targets, lse, dloss, torch.empty_like(h) if wide else None, torch.empty_like(w, dtype=F32))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("std", [3.0, 30.0])
def test_steep_softmax(ra, dtype, std):
    # logits of hundreds: a few words have all the probability
    gpu()
    rows, cols, vocab = 260, 64, 3000
    gen = generator(11)
    h, w = matrix(rows, cols, dtype, gen), matrix(vocab, cols, dtype, gen, std=std)
    check_both(ra, h, w, draw_targets(rows, vocab, gen), torch.rand(rows, generator=gen, device="cuda"))


@pytest.mark.gpu
def test_logits_of_minus_infinity(ra):
    # one word's logits overflow downwards: its probability is 0 and so is its gradient
    gpu()
    rows, cols, vocab = 40, 64, 700
    gen = generator(12)
    h, w = matrix(rows, cols, BF16, gen), matrix(vocab, cols, BF16, gen, std=0.1)
    h[:, 0] = 2.0 ** 120
    w[:, 0] = 0
    for dead in (range(300, 301), range(256, 512), range(0, 699)):
        w[:, 0] = 0
        w[dead.start:dead.stop, 0] = -(2.0 ** 120)
        live = [v for v in range(vocab) if v not in dead]
        targets = torch.tensor(live, device="cuda")[torch.randint(0, len(live), (rows,), generator=gen, device="cuda")]
        loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        ra.ra_cross_entropy_forward(h, w, targets, loss, lse, workspace=scratch(ra, h, w))
        logits = (h[:, 1:].double() @ w[live, 1:].double().t())
        assert_within(lse, torch.logsumexp(logits, 1), torch.full((rows,), 1e-4, dtype=torch.float64, device="cuda"), "lse")
        dh, dw = torch.empty_like(h), torch.empty_like(w)
        ra.ra_cross_entropy_backward(h, w, targets, lse, None, dh, dw, workspace=scratch(ra, h, w, backward=True))
        assert (dw[dead.start:dead.stop] == 0).all() and torch.isfinite(dw[:, 1:]).all() and torch.isfinite(dh[:, 1:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_targets_outside_the_vocabulary_and_nan(ra, dtype):
    gpu()
    rows, cols, vocab = 300, 72, 500
    gen = generator(13)
    h, w = matrix(rows, cols, dtype, gen), matrix(vocab, cols, dtype, gen, std=0.1)
    targets = draw_targets(rows, vocab, gen, I64, [1, 2])
    bad = [0, 7, 255, 299]
    for i, v in zip(bad, (vocab, -1, 2 ** 40 + 3, -2 ** 63)):
        targets[i] = v
    h[17, 5] = float("nan")
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ra.ra_cross_entropy_forward(h, w, targets, loss, lse, workspace=scratch(ra, h, w))
    wrong = torch.zeros(rows, dtype=torch.bool, device="cuda")
    wrong[bad + [17]] = True
    assert torch.isnan(loss[wrong]).all() and torch.isnan(lse[wrong]).all()
    assert torch.isfinite(loss[~wrong]).all() and torch.isfinite(lse[~wrong]).all()
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    ra.ra_cross_entropy_backward(h, w, targets, torch.nan_to_num(lse), None, dh, dw, workspace=scratch(ra, h, w, backward=True))
    assert torch.isnan(dh[wrong]).all() and torch.isfinite(dh[~wrong]).all() and torch.isnan(dw).all()
    # a gradient that is not finite reaches its own row, and the weight's gradient
    targets = draw_targets(rows, vocab, gen)
    h[17, 5] = 0
    check_forward(ra, h, w, targets, loss, lse)
    dloss = torch.ones(rows, device="cuda")
    dloss[20], dloss[21] = float("inf"), float("nan")
    ra.ra_cross_entropy_backward(h, w, targets, lse, dloss, dh, dw, workspace=scratch(ra, h, w, backward=True))
    fine = torch.ones(rows, dtype=torch.bool, device="cuda")
    fine[20:22] = False
    assert torch.isfinite(dh[fine]).all() and not torch.isfinite(dh[~fine]).any() and not torch.isfinite(dw).any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rows,cols,vocab", [(BF16, 8192, 64, 40001), (F16, 30000, 40, 9000), (BF16, 3000, 512, 130_000)])
def test_several_pieces(ra, dtype, rows, cols, vocab):
    # more than one piece of g
    gpu()
    gen = generator(rows)
    h, w = matrix(rows, cols, dtype, gen), matrix(vocab, cols, dtype, gen, std=1.0 / cols ** 0.5)
    targets = draw_targets(rows, vocab, gen, I32, range(0, rows, 9))
    lse = check_forward(ra, h, w, targets)
    dloss = torch.rand(rows, generator=gen, device="cuda") / rows
    dh, dw = torch.empty_like(h), matrix(vocab, cols, dtype, gen, std=1e-3)
    check_backward(ra, h, w, targets, lse, dloss, dh, dw, accumulate=True)


@pytest.mark.gpu
def test_no_rows(ra):
    gpu()
    h, t, none = torch.empty(0, 16, dtype=BF16, device="cuda"), torch.empty(0, dtype=I64, device="cuda"), torch.empty(0, device="cuda")
    w = torch.ones(30, 16, dtype=BF16, device="cuda")
    dw = torch.ones_like(w)
    ws = torch.empty(ra.ra_cross_entropy_workspace(h, w, backward=True), dtype=torch.uint8, device="cuda")
    ra.ra_cross_entropy_forward(h, w, t, none, none, workspace=ws)
    ra.ra_cross_entropy_backward(h, w, t, none, None, h, dw, accumulate=True, workspace=ws)
    assert (dw == 1).all()
    ra.ra_cross_entropy_backward(h, w, t, none, None, h, dw, workspace=ws)
    assert (dw == 0).all()


@pytest.mark.gpu
def test_against_differences(ra):
    # along random directions, d/ds sum(dloss * loss(s)) by central differences of the 64-bit formula
    gpu()
    rows, cols, vocab = 50, 64, 200
    gen = generator(15)
    h, w = matrix(rows, cols, F16, gen), matrix(vocab, cols, F16, gen, std=0.2)
    targets = draw_targets(rows, vocab, gen, I64, [3, 4])
    counts = targets != IGNORE
    dloss = torch.rand(rows, generator=gen, device="cuda")
    lse = check_forward(ra, h, w, targets)
    dh, dw = torch.empty_like(h), torch.empty_like(w, dtype=F32)
    ra.ra_cross_entropy_backward(h, w, targets, lse, dloss, dh, dw, workspace=scratch(ra, h, w, backward=True))

    def value(h64, w64):
        each = torch.nn.functional.cross_entropy(h64[counts] @ w64.t(), targets[counts], reduction="none")
        return float((each * dloss.double()[counts]).sum())

    step = 1e-4
    for grad, at in ((dh, 0), (dw, 1)):
        args = [h.double(), w.double()]
        d = torch.randn(args[at].shape, generator=gen, dtype=torch.float64, device="cuda")
        plus, minus = list(args), list(args)
        plus[at], minus[at] = args[at] + step * d, args[at] - step * d
        want = (value(*plus) - value(*minus)) / (2 * step)
        terms = grad.double() * d
        # g and the stored gradient are each off by 2^-11 of themselves, the sums by a few hundred u
        assert abs(float(terms.sum()) - want) <= 4 * 2.0 ** -11 * float(terms.abs().sum()) + 1e3 * step * step * float(terms.abs().sum())


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 40, 700])
def test_same_bits_again_on_another_stream_and_in_a_graph(ra, rows):
    gpu()
    cols, vocab = 128, 3000
    gen = generator(16)
    h, w = matrix(rows, cols, BF16, gen), matrix(vocab, cols, BF16, gen, std=0.1)
    targets = draw_targets(rows, vocab, gen, I64, range(1, rows, 5))
    ws = scratch(ra, h, w, backward=True)
    fs = scratch(ra, h, w)

    def both(o, stream=None):
        ra.ra_cross_entropy_forward(h, w, targets, o[0], o[1], workspace=fs, stream=stream)
        ra.ra_cross_entropy_backward(h, w, targets, o[1], o[0], o[2], o[3], workspace=ws, stream=stream)

    def outputs():
        return [torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda"), torch.zeros_like(h), torch.zeros_like(w)]

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
    assert (got[1] == 0).all()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_more_than_32_bits_of_elements(ra):
    # a head of 2.2e9 elements: words at both ends
    gpu()
    cols = 8192
    vocab = (1 << 31) // cols + 301
    gen = generator(17)
    rows = 5
    h = matrix(rows, cols, BF16, gen)
    w = torch.empty(vocab, cols, dtype=BF16, device="cuda")
    for a in range(0, vocab, 16384):
        w[a:a + 16384].normal_(generator=gen, std=0.01)
    targets = torch.tensor([0, vocab - 1, vocab // 2, vocab - 2, 1], device="cuda")
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ra.ra_cross_entropy_forward(h, w, targets, loss, lse, workspace=scratch(ra, h, w))
    logits = torch.cat([h.double() @ w[a:a + 16384].double().t() for a in range(0, vocab, 16384)], 1)
    want = torch.logsumexp(logits, 1)
    # 2 cols u sum|h w| is 2 * 8192 * 2^-24 * 8192 * 0.8 * 0.008 = 0.05 at most; the sums' errors are random, 1e-3 is 1/50
    tol = torch.full((rows,), 1e-3, dtype=torch.float64, device="cuda")
    assert_within(lse, want, tol, "lse")
    assert_within(loss, want - logits.gather(1, targets[:, None])[:, 0], 2 * tol, "loss")
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    ra.ra_cross_entropy_backward(h, w, targets, lse, None, dh, dw, workspace=scratch(ra, h, w, backward=True))
    p = torch.exp(logits - lse.double()[:, None])
    p[torch.arange(rows, device="cuda"), targets] -= 1
    dh_want = sum(p[:, a:a + 16384] @ w[a:a + 16384].double() for a in range(0, vocab, 16384))
    size = sum(p[:, a:a + 16384].abs() @ w[a:a + 16384].double().abs() for a in range(0, vocab, 16384))
    assert_within(dh, dh_want, 2.0 ** -8 * dh_want.abs() + (2.0 ** -8 + 2e-3) * size, "dhidden")
    for part in (slice(0, 64), slice(vocab // 2 - 32, vocab // 2 + 32), slice(vocab - 64, vocab)):
        want = p[:, part].t() @ h.double()
        size = p[:, part].abs().t() @ h.double().abs()
        assert_within(dw[part], want, 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2e-3) * size, "dweight")


# Fake addresses that are never dereferenced: every case is refused on the host.
BASE = 0x7F0000000000
MB = 1 << 20


def test_forward_refusals(ra):
    need = ra.lib().ra_cross_entropy_workspace(BASE, 64, 16, 64, 100, 2, 0)

    def call(h=BASE, hs=64, w=BASE + 2 * MB, ws=64, t=BASE + 4 * MB, size=8, loss=BASE + 5 * MB, lse=BASE + 6 * MB, rows=16, cols=64, vocab=100,
             dt=2, scratch=BASE + 8 * MB, n=need):
        return ra.lib().ra_cross_entropy_forward(h, hs, w, ws, t, size, -100, loss, lse, rows, cols, vocab, dt, scratch, n, None)

    bad, alias = ra.RA_ERR_INVALID_ARG, ra.RA_ERR_ALIAS
    assert call(dt=0) == call(dt=3) == ra.RA_ERR_UNSUPPORTED and call(dt=8) == bad
    assert call(size=2) == call(hs=63) == call(ws=63) == call(cols=0) == call(vocab=0) == bad
    assert call(h=0) == call(w=0) == call(t=0) == call(loss=0) == call(lse=0) == call(scratch=0) == bad
    assert call(h=BASE + 1) == call(t=BASE + 4 * MB + 4) == call(loss=BASE + 5 * MB + 2) == call(scratch=BASE + 8 * MB + 8) == bad
    assert call(n=need - 1) == call(rows=1 << 31) == call(vocab=1 << 31) == call(rows=1 << 30, cols=1 << 30, hs=1 << 30, ws=1 << 30) == bad
    wide = (1 << 24) + 1
    assert call(rows=1, vocab=1, cols=wide, hs=wide, ws=wide, w=BASE + 64 * MB, t=BASE + 128 * MB, loss=BASE + 129 * MB, lse=BASE + 130 * MB,
                scratch=BASE + 256 * MB, n=1 << 40) == bad
    assert call(loss=BASE) == call(lse=BASE + 5 * MB + 4) == call(scratch=BASE + 2 * MB) == call(loss=BASE + 4 * MB) == alias
    assert call(rows=0) == ra.RA_SUCCESS


def test_backward_refusals(ra):
    need = ra.lib().ra_cross_entropy_workspace(BASE, 64, 16, 64, 100, 2, 1)

    def call(h=BASE, hs=64, w=BASE + 2 * MB, ws=64, t=BASE + 4 * MB, size=8, lse=BASE + 6 * MB, dl=BASE + 7 * MB, dh=BASE + 8 * MB, dhs=64,
             dw=BASE + 10 * MB, dws=64, acc=0, rows=16, cols=64, vocab=100, dt=2, wdt=0, scratch=BASE + 16 * MB, n=need):
        return ra.lib().ra_cross_entropy_backward(h, hs, w, ws, t, size, -100, lse, dl, dh, dhs, dw, dws, acc, rows, cols, vocab, dt, wdt,
                                                  scratch, n, None)

    bad, alias = ra.RA_ERR_INVALID_ARG, ra.RA_ERR_ALIAS
    assert call(dt=0) == call(wdt=3) == call(wdt=1) == ra.RA_ERR_UNSUPPORTED and call(wdt=9) == bad
    assert call(size=1) == call(hs=63) == call(ws=63) == call(dhs=63) == call(dws=63) == call(cols=0) == call(vocab=0) == bad
    assert call(h=0) == call(w=0) == call(t=0) == call(lse=0) == call(scratch=0) == call(n=need - 1) == bad
    assert call(dw=BASE + 10 * MB + 2) == call(dh=BASE + 8 * MB + 1) == call(dl=BASE + 7 * MB + 1) == bad
    assert call(dh=BASE) == call(dh=BASE + 2) == call(dw=BASE + 2 * MB) == call(dw=BASE + 8 * MB) == call(scratch=BASE) == alias
    assert call(dh=BASE + 6 * MB) == call(dw=BASE + 4 * MB) == call(scratch=BASE + 7 * MB) == alias
    assert call(dh=0, dw=0) == call(rows=0, acc=1) == call(rows=0, dw=0) == ra.RA_SUCCESS


def test_workspace_sizes(ra):
    def size(rows, cols, vocab, backward=0, w=BASE, stride=None, dt=2):
        return ra.lib().ra_cross_entropy_workspace(w, cols if stride is None else stride, rows, cols, vocab, dt, backward)

    assert size(8, 1 << 24, 8) > 0
    assert size(1 << 31, 8, 8) == size(8, 8, 1 << 31) == size(8, (1 << 24) + 1, 8) == size(8, 8, 8, dt=0) == size(8, 8, 8, dt=3) == 0
    copy = 50257 * 1024 * 2
    assert size(64, 1024, 50257, w=BASE + 2) - size(64, 1024, 50257) >= copy  # not on a 16-byte boundary: a copy of the weight
    assert size(64, 1024, 50257, stride=1025) - size(64, 1024, 50257) >= copy
    assert size(64, 1024, 50257, w=BASE + 32, stride=1032) == size(64, 1024, 50257)
    # two pieces of g, not all of it: at most 192 MiB each, or 1024 columns
    assert size(8192, 1024, 50257, 1) < 8192 * 50257 * 2
    assert size(1 << 20, 64, 50257, 1) < 2 * (1 << 20) * 1024 * 2 + (1 << 20) * 64 * 8


def test_binding_refusals(ra):
    h, w, t, f = torch.zeros(4, 8, dtype=BF16), torch.zeros(9, 8, dtype=BF16), torch.zeros(4, dtype=I64), torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_cross_entropy_forward(h, w, t, f, f, workspace=f)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_cross_entropy_backward(h, w, t, f, f, h, w, workspace=f)
    with pytest.raises(ValueError, match="two dimensions"):
        ra.ra_cross_entropy_forward(h[0], w, t, f, f, workspace=f)
