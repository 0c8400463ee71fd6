"""ra_layernorm_forward / ra_layernorm_backward against the formulas in 64 bits.

Tolerances come from the arithmetic, before any run. With u = 2^-24 a sum of n
fp32 terms taken as chains of at most n/32 terms joined by trees is off by at
most k u sum|term|, k = n/32 + 32 (the tree, the products and the scalar
operations around it in the 32); a stored result adds half an ulp of its type
(2^-24, 2^-11, 2^-8 relative; fp16's smallest step is 2^-24)."""

import ctypes

import pytest
import torch

U = 2.0 ** -24
ROUND = {torch.float32: U, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
STEP = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-5


@pytest.fixture(scope="module")
def ra():
    from ring_all_reduce_02_gb300 import build, ra as binding

    build.build()
    return binding


def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def matrix(rows, cols, dtype, gen, std=1.0, offset=0.0, pad=0, shift=0):
    """A [rows, cols] view with `pad` elements between rows, `shift` elements past an allocation's start."""
    stride = cols + pad
    base = torch.full((rows * stride + shift + 1,), 7.0, dtype=dtype, device="cuda")
    v = base[shift:].as_strided((rows, cols), (stride, 1))
    v.copy_(torch.randn(rows, cols, generator=gen, dtype=torch.float64) * std + offset)
    return v


def forward64(x, w, b, eps=EPS):
    x = x.double().cpu()
    mean = x.mean(1, keepdim=True)
    rstd = ((x - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    h = (x - mean) * rstd
    w = torch.ones(x.shape[1], dtype=torch.float64) if w is None else w.double().cpu()
    b = torch.zeros(x.shape[1], dtype=torch.float64) if b is None else b.double().cpu()
    return x, mean, rstd, h, w, b


def assert_within(got, want, tol, what):
    got = got.double().cpu()
    assert got.shape == want.shape
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = (got - want).abs() - tol
    assert (bad <= 0).all(), f"{what}: off by {float((got - want).abs().max())}, {float(bad.max())} over the bound"


def check_forward(ra, x, w, b, y, mean, rstd, eps=EPS):
    x64, m64, r64, h, w64, b64 = forward64(x, w, b, eps)  # before the call: y may be x
    rows, cols = x64.shape
    ra.ra_layernorm_forward(x, w, b, y, mean, rstd, eps=eps)
    torch.cuda.synchronize()
    k = (cols / 32 + 32) * U
    top = x64.abs().amax(1, keepdim=True)
    want = h * w64 + b64
    # the mean is off by k u max|x|, the deviation relatively by 2 k u and by the mean's own error, and so xhat
    dh = k * (3 * h.abs() + 3 * top * r64)
    assert_within(y, want, ROUND[y.dtype] * want.abs() + STEP[y.dtype] + 1.01 * (w64.abs() * dh + 2 * U * want.abs()), "y")
    if mean is not None:
        assert_within(mean, m64[:, 0], k * top[:, 0] + U * m64[:, 0].abs(), "mean")
    if rstd is not None:
        assert_within(rstd, r64[:, 0], r64[:, 0] * k * (3 + 3 * (top * r64)[:, 0]), "rstd")


def check_backward(ra, dy, x, w, mean, rstd, dx, dw, db, accumulate=False, workspace=None):
    rows, cols = x.shape
    dy64, x64 = dy.double().cpu(), x.double().cpu()
    m64, r64 = mean.double().cpu()[:, None], rstd.double().cpu()[:, None]
    w64 = torch.ones(cols, dtype=torch.float64) if w is None else w.double().cpu()
    old = [None if t is None else t.double().cpu() for t in (dw, db)]
    h, a = (x64 - m64) * r64, dy64 * w64
    c1, c2 = a.mean(1, keepdim=True), (a * h).mean(1, keepdim=True)
    want = r64 * (a - c1 - h * c2)
    if workspace is None:
        workspace = torch.empty(max(1, ra.ra_layernorm_workspace(rows, cols)), dtype=torch.uint8, device="cuda")
        workspace.fill_(255)  # NaN: its contents do not matter
    ra.ra_layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, workspace=workspace, accumulate=accumulate)
    torch.cuda.synchronize()
    k = (cols / 32 + 32) * U
    dh = 4 * U * (x64.abs() + m64.abs()) * r64
    abs_ah = (a * h).abs().mean(1, keepdim=True) + (a.abs() * dh).mean(1, keepdim=True)
    tol = r64 * (k * (a.abs() + a.abs().mean(1, keepdim=True) + 2 * h.abs() * abs_ah)
                 + dh * abs_ah + h.abs() * (a.abs() * dh).mean(1, keepdim=True))
    assert_within(dx, want, ROUND[dx.dtype] * want.abs() + STEP[dx.dtype] + 1.01 * tol, "dx")
    for got, term, extra, name, was in ((dw, dy64 * h, dy64.abs() * dh, "dw", old[0]), (db, dy64, 0 * dy64, "db", old[1])):
        if got is None:
            continue
        want = term.sum(0) + (was if accumulate else 0)
        # any order of a sum of `rows` terms: rows u sum|term|
        tol = (rows + 8) * U * (term.abs().sum(0) + want.abs()) + extra.sum(0)
        assert_within(got, want, ROUND[got.dtype] * want.abs() + STEP[got.dtype] + 1.01 * tol, name)


SHAPES = [(1, 1), (3, 1), (1, 2), (5, 31), (1, 1024), (7, 33), (64, 64), (33, 100), (19, 1000), (40, 1024), (9, 1023),
          (300, 768), (7, 1537), (5, 2048), (3, 4095), (4, 4096), (2, 5000), (3, 8192), (2, 8193), (3, 12290), (2, 16384),
          (2, 20000), (1, 33001), (2, 70000)]
TYPES = [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,wdtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward_and_backward(ra, rows, cols, dtype, wdtype):
    gpu()
    gen = torch.Generator().manual_seed(rows * 100003 + cols)
    x = matrix(rows, cols, dtype, gen, std=2.0, offset=0.7)
    w = (torch.randn(cols, generator=gen) * 0.3 + 1).to(wdtype).cuda()
    b = (torch.randn(cols, generator=gen) * 0.3).to(wdtype).cuda()
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    check_forward(ra, x, w, b, torch.empty_like(x), mean, rstd)
    dy = matrix(rows, cols, dtype, gen, std=0.1)
    check_backward(ra, dy, x, w, mean, rstd, torch.empty_like(x), torch.empty_like(w), torch.empty_like(w))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (F16, F32), (F32, F32)])
@pytest.mark.parametrize("cols,pad,shift", [(64, 8, 0), (256, 3, 0), (1024, 1, 1), (1024, 0, 1), (1000, 24, 4), (2048, 2, 2),
                                            (4096, 0, 3), (4097, 15, 0), (9000, 8, 8)])
def test_strides_and_alignment(ra, dtype, wdtype, cols, pad, shift):
    gpu()
    rows = 21
    gen = torch.Generator().manual_seed(cols + 31 * pad + shift)
    x = matrix(rows, cols, dtype, gen, pad=pad, shift=shift)
    w = matrix(1, cols, wdtype, gen, shift=shift)[0]
    b = matrix(1, cols, wdtype, gen, shift=1)[0]
    y = matrix(rows, cols, dtype, gen, pad=pad + 2, shift=0)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    check_forward(ra, x, w, b, y, mean, rstd)
    dy = matrix(rows, cols, dtype, gen, pad=0, shift=shift)
    dx = matrix(rows, cols, dtype, gen, pad=pad, shift=1)
    check_backward(ra, dy, x, w, mean, rstd, dx, matrix(1, cols, wdtype, gen, shift=1)[0],
                   matrix(1, cols, wdtype, gen, shift=shift)[0])
    # what lies between the rows is left alone
    for t in (y, dx):
        flat = t.as_strided((rows - 1, t.stride(0) - cols), (t.stride(0), 1), t.storage_offset() + cols)
        assert (flat == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [96, 1024, 1025, 6000, 40000])
def test_in_place_and_optional_buffers(ra, cols):
    gpu()
    rows = 37
    gen = torch.Generator().manual_seed(cols)
    x = matrix(rows, cols, BF16, gen)
    w, b = matrix(1, cols, F32, gen)[0], matrix(1, cols, F32, gen)[0]
    check_forward(ra, x, None, None, torch.empty_like(x), None, None)
    check_forward(ra, x, w, None, torch.empty_like(x), None, None)
    check_forward(ra, x, None, b, torch.empty_like(x), torch.empty(rows, device="cuda"), None)
    y = x.clone()
    check_forward(ra, y, w, b, y, None, None)  # in place
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ra.ra_layernorm_forward(x, w, b, torch.empty_like(x), mean, rstd)
    dy = matrix(rows, cols, BF16, gen)
    check_backward(ra, dy, x, None, mean, rstd, torch.empty_like(x), None, None)
    check_backward(ra, dy, x, w, mean, rstd, torch.empty_like(x), None, torch.empty_like(w))
    check_backward(ra, dy, x, w, mean, rstd, torch.empty_like(x), torch.ones_like(w), None, accumulate=True)
    in_dy, in_x = dy.clone(), x.clone()
    check_backward(ra, in_dy, x, w, mean, rstd, in_dy, torch.empty_like(w), torch.empty_like(w))
    check_backward(ra, dy, in_x, w, mean, rstd, in_x, torch.ones_like(w), torch.ones_like(w), accumulate=True)


@pytest.mark.gpu
def test_large_offset_keeps_the_deviation(ra):
    # mean 300 times the deviation: a difference of raw moments would leave 7 bits
    gpu()
    gen = torch.Generator().manual_seed(1)
    for cols in (500, 1024, 4096, 70001):
        x = matrix(5, cols, F32, gen, std=1.0, offset=300.0)
        check_forward(ra, x, None, None, torch.empty_like(x), torch.empty(5, device="cuda"), torch.empty(5, device="cuda"))
        # a constant row: the deviation is 0, y the bias
        x.fill_(3.0)
        b = matrix(1, cols, F32, gen)[0]
        y = torch.empty_like(x)
        ra.ra_layernorm_forward(x, None, b, y)
        assert torch.equal(y, b.expand_as(y))


@pytest.mark.gpu
def test_non_finite_rows_stay_their_own(ra):
    gpu()
    gen = torch.Generator().manual_seed(2)
    for cols in (64, 1024, 5000):
        x = matrix(6, cols, F16, gen)
        clean = x.clone()
        x[1, cols // 2] = float("inf")
        x[4, 0] = float("nan")
        y, want = torch.empty_like(x), torch.empty_like(x)
        ra.ra_layernorm_forward(x, None, None, y)
        ra.ra_layernorm_forward(clean, None, None, want)
        assert torch.isnan(y[4]).all() and torch.isnan(y[1]).any()
        for r in (0, 2, 3, 5):
            assert torch.equal(y[r], want[r])


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(1, 64), (2, 1000), (151, 128), (153, 1024), (5000, 256), (100001, 48), (20011, 2050),
                                       (3001, 9001)])
def test_weight_gradient_counts_every_row_once(ra, rows, cols):
    # mean 0, rstd 1 and small whole numbers: the column sums are exact whatever their order
    gpu()
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randint(-3, 4, (rows, cols), generator=gen, device="cuda").to(BF16)
    dy = torch.randint(-3, 4, (rows, cols), generator=gen, device="cuda").to(BF16)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dw, db = torch.full((cols,), 5.0, device="cuda"), torch.full((cols,), -5.0, device="cuda")
    ws = torch.empty(ra.ra_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda").fill_(255)
    dx = torch.empty_like(x)
    for accumulate, times in ((False, 1), (True, 2)):
        ra.ra_layernorm_backward(dy, x, None, mean, rstd, dx, dw, db, workspace=ws, accumulate=accumulate)
        assert torch.equal(dw.double(), times * (dy.double() * x.double()).sum(0))
        assert torch.equal(db.double(), times * dy.double().sum(0))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 20000), (75, 20000), (77, 18001), (701, 17000), (1003, 32768), (613, 12289), (90, 32769)])
def test_rows_shared_by_several_ctas(ra, rows, cols, dtype):
    gpu()
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randint(-3, 4, (rows, cols), generator=gen, device="cuda").to(dtype)
    dy = torch.randint(-3, 4, (rows, cols), generator=gen, device="cuda").to(dtype)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    w = torch.ones(cols, device="cuda")
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(ra.ra_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda").fill_(255)
    ra.ra_layernorm_backward(dy, x, w, mean, rstd, torch.empty_like(x), dw, db, workspace=ws)
    assert torch.equal(dw.double(), (dy.double() * x.double()).sum(0))  # whole numbers: exact in any order
    assert torch.equal(db.double(), dy.double().sum(0))
    few = min(rows, 120)
    x = (torch.randn(few, cols, generator=gen, device="cuda") * 2 + 0.7).to(dtype)
    dy = (torch.randn(few, cols, generator=gen, device="cuda") * 0.1).to(dtype)
    w = torch.randn(cols, generator=gen, device="cuda") * 0.3 + 1
    mean, rstd = mean[:few].clone(), rstd[:few].clone()
    ra.ra_layernorm_forward(x, w, None, torch.empty_like(x), mean, rstd)
    check_backward(ra, dy, x, w, mean, rstd, torch.empty_like(x), dw, db)


@pytest.mark.gpu
def test_no_rows(ra):
    gpu()
    x = torch.empty(0, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    none = torch.empty(0, device="cuda")
    ra.ra_layernorm_forward(x, w, w, x, none, none)
    dw, db = torch.ones(16, device="cuda"), torch.ones(16, device="cuda")
    ra.ra_layernorm_backward(x, x, w, none, none, x, dw, db, workspace=torch.empty(0, device="cuda"), accumulate=True)
    assert (dw == 1).all() and (db == 1).all()
    ra.ra_layernorm_backward(x, x, w, none, none, x, dw, db, workspace=torch.empty(0, device="cuda"))
    assert (dw == 0).all() and (db == 0).all()
    ra.ra_layernorm_forward(torch.empty(4, 0, device="cuda"), None, None, torch.empty(4, 0, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [40, 1024, 3000])
def test_backward_against_differences(ra, cols):
    # along random directions, d/dt sum(dy * y(t)) by central differences of the 64-bit forward pass
    gpu()
    rows = 6
    gen = torch.Generator().manual_seed(cols)
    x, dy = matrix(rows, cols, F32, gen), matrix(rows, cols, F32, gen)
    w, b = matrix(1, cols, F32, gen, offset=1.0)[0], matrix(1, cols, F32, gen)[0]
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ra.ra_layernorm_forward(x, w, b, torch.empty_like(x), mean, rstd)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(ra.ra_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    ra.ra_layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, workspace=ws)

    def loss(x, w, b):
        _, _, _, h, w, b = forward64(x, w, b)
        return float(((h * w + b) * dy.double().cpu()).sum())

    t = 1e-4
    for grad, at in ((dx, 0), (dw, 1), (db, 2)):
        args = [v.double().cpu() for v in (x, w, b)]
        d = torch.randn(args[at].shape, generator=gen, dtype=torch.float64)
        plus, minus = list(args), list(args)
        plus[at], minus[at] = args[at] + t * d, args[at] - t * d
        want = (loss(*plus) - loss(*minus)) / (2 * t)
        terms = grad.double().cpu() * d
        # the fp32 gradient is off by a few hundred u at most, the differences by t^2 times the third derivative
        assert abs(float(terms.sum()) - want) <= 300 * U * float(terms.abs().sum()) + 1e3 * t * t * float(terms.abs().sum())


@pytest.mark.gpu
def test_another_stream_and_a_graph(ra):
    gpu()
    gen = torch.Generator().manual_seed(9)
    rows, cols = 700, 1024
    x, dy = matrix(rows, cols, BF16, gen), matrix(rows, cols, BF16, gen)
    w = matrix(1, cols, BF16, gen)[0]
    ws = torch.empty(ra.ra_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")

    def outputs():
        return [torch.zeros_like(x), torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda"), torch.zeros_like(x),
                torch.zeros_like(w), torch.zeros_like(w)]

    def both(o, stream=None):
        ra.ra_layernorm_forward(x, w, w, o[0], o[1], o[2], stream=stream)
        ra.ra_layernorm_backward(dy, x, w, o[1], o[2], o[3], o[4], o[5], workspace=ws, stream=stream)

    want, got = outputs(), outputs()
    both(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
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
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [4096, 4095])
def test_more_than_32_bits_of_elements(ra, cols):
    # 4.4e9 elements: the last rows against the formula, and the weight gradients see them
    gpu()
    rows, tail = (1 << 32) // cols + 20011, 300
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.ones(rows, cols, dtype=BF16, device="cuda")
    x[-tail:] = torch.randn(tail, cols, generator=gen, device="cuda").to(BF16)
    w = torch.randn(cols, generator=gen, device="cuda").to(BF16)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ra.ra_layernorm_forward(x, w, w, y, mean, rstd)
    x64, m64, r64, h, w64, b64 = forward64(x[-tail:], w, w)
    k = (cols / 32 + 32) * U
    top = x64.abs().amax(1, keepdim=True)
    want = h * w64 + b64
    assert_within(y[-tail:], want, ROUND[BF16] * want.abs() + 1.01 * (w64.abs() * k * (3 * h.abs() + 3 * top * r64) + 2 * U * want.abs()), "y")
    assert_within(mean[-tail:], m64[:, 0], k * top[:, 0] + U * m64[:, 0].abs(), "mean")
    assert torch.equal(y[0], w) and torch.equal(y[rows // 2], w)  # constant rows give the bias
    dy = y.zero_()
    dy[-tail:] = torch.randint(-3, 4, (tail, cols), generator=gen, device="cuda").to(BF16)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w, dtype=F32), torch.empty_like(w, dtype=F32)
    ws = torch.empty(ra.ra_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    ra.ra_layernorm_backward(dy, x, w.float(), mean, rstd, dx, dw, db, workspace=ws)
    assert torch.equal(db.double(), dy[-tail:].double().sum(0)) and (dx[0] == 0).all() and (dx[rows // 2] == 0).all()
    h = (x64 - mean[-tail:].double().cpu()[:, None]) * rstd[-tail:].double().cpu()[:, None]
    terms = dy[-tail:].double().cpu() * h
    assert_within(dw, terms.sum(0), (tail + 16) * U * terms.abs().sum(0) + U, "dw")
    a = dy[-tail:].double().cpu() * w64
    want = rstd[-tail:].double().cpu()[:, None] * (a - a.mean(1, keepdim=True) - h * (a * h).mean(1, keepdim=True))
    tol = 4 * k * r64 * (a.abs() + a.abs().mean(1, keepdim=True) + 2 * h.abs() * (a * h).abs().mean(1, keepdim=True))
    assert_within(dx[-tail:], want, ROUND[BF16] * want.abs() + tol, "dx")


# Fake addresses that are never dereferenced: every case is refused on the host.
BASE = 0x7F0000000000
MB = 1 << 20


def test_forward_refusals(ra):
    def call(x=BASE, xs=64, w=BASE + 4 * MB, b=BASE + 5 * MB, y=BASE + 8 * MB, ys=64, mean=BASE + 12 * MB, rstd=BASE + 13 * MB,
             rows=16, cols=64, eps=1e-5, dt=2, wdt=0):
        return ra.lib().ra_layernorm_forward(x, xs, w, b, y, ys, mean, rstd, rows, cols, eps, dt, wdt, None)

    bad, alias = ra.RA_ERR_INVALID_ARG, ra.RA_ERR_ALIAS
    assert call(dt=3) == call(wdt=3) == ra.RA_ERR_UNSUPPORTED
    assert call(dt=7) == call(wdt=-1) == bad
    assert call(dt=2, wdt=1) == call(dt=0, wdt=2) == ra.RA_ERR_UNSUPPORTED
    assert call(x=0) == call(y=0) == bad
    assert call(x=BASE + 1) == call(y=BASE + 8 * MB + 1) == call(w=BASE + 4 * MB + 2) == call(mean=BASE + 12 * MB + 2) == bad
    assert call(xs=63) == call(ys=63) == bad
    assert call(eps=-1.0) == call(eps=float("nan")) == call(eps=float("inf")) == bad
    assert call(rows=1 << 40, cols=1 << 30, xs=1 << 30, ys=1 << 30) == bad
    assert call(y=BASE + 2) == call(y=BASE, ys=65) == call(y=BASE + 4 * MB - 2) == alias
    assert call(mean=BASE + 13 * MB - 4) == call(rstd=BASE) == call(mean=BASE + 8 * MB) == alias
    assert call(rows=0) == call(cols=0, xs=0, ys=0) == ra.RA_SUCCESS


def test_backward_refusals(ra):
    def call(dy=BASE, dys=64, x=BASE + 2 * MB, xs=64, w=BASE + 4 * MB, mean=BASE + 5 * MB, rstd=BASE + 6 * MB, dx=BASE + 8 * MB,
             dxs=64, dw=BASE + 10 * MB, db=BASE + 11 * MB, acc=0, rows=16, cols=64, dt=2, wdt=0, ws=BASE + 12 * MB, nws=None):
        nws = ra.ra_layernorm_workspace(16, 64) if nws is None else nws
        return ra.lib().ra_layernorm_backward(dy, dys, x, xs, w, mean, rstd, dx, dxs, dw, db, acc, rows, cols, dt, wdt, ws, nws,
                                              None)

    bad, alias = ra.RA_ERR_INVALID_ARG, ra.RA_ERR_ALIAS
    assert ra.ra_layernorm_workspace(16, 64) > 0 and ra.ra_layernorm_workspace(0, 64) == 0
    assert call(dt=3) == call(dt=1, wdt=2) == ra.RA_ERR_UNSUPPORTED
    assert call(dy=0) == call(x=0) == call(mean=0) == call(rstd=0) == call(dx=0) == bad
    assert call(ws=0) == call(nws=0) == call(ws=BASE + 12 * MB + 4) == bad
    assert call(dys=63) == call(xs=1) == call(dxs=0) == bad
    assert call(dw=BASE + 10 * MB + 1) == call(dx=BASE + 8 * MB + 1) == bad
    assert call(dx=BASE + 2) == call(dx=BASE, dxs=65) == call(dw=BASE + 4 * MB) == call(db=BASE + 10 * MB) == alias
    assert call(ws=BASE + 8 * MB) == call(ws=BASE) == alias
    assert call(rows=0, acc=1) == call(cols=0) == ra.RA_SUCCESS


def test_binding_refusals(ra):
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_layernorm_forward(x, None, None, x)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_layernorm_backward(x, x, None, x[:, 0], x[:, 0], x)
    assert isinstance(ctypes.sizeof(ra.AdamwTensor), int)
