"""What layer norm owes to rows that lie far from zero, and to every row of a call.

Tolerances as in test_layernorm.py, with u = 2^-24, but xhat = (x - mean) rstd
is held to its own two roundings (3 u |xhat|) wherever the row lies: no term in
|mean|. Everything is compared in 64 bits on the GPU."""

import pytest
import torch

import test_layernorm
from test_layernorm import BF16, EPS, F16, F32, ROUND, STEP, U, gpu

CONST_RSTD = EPS ** -0.5


@pytest.fixture(scope="module")
def ra():
    from ring_all_reduce_02_gb300 import build, ra as binding

    build.build()
    return binding


def within(got, want, tol, what):
    bad = (got.double() - want).abs() - tol
    assert not torch.isnan(got).any() and bool((bad <= 0).all()), f"{what}: {float(bad.max())} over the bound"


def backward(ra, dy, x, w, mean, rstd, dx=None, wdtype=F32):
    rows, cols = x.shape
    dx = torch.empty_like(x) if dx is None else dx
    dw, db = (torch.empty(cols, dtype=wdtype, device="cuda") for _ in range(2))
    ws = torch.empty(max(1, ra.ra_layernorm_workspace(rows, cols)), dtype=torch.uint8, device="cuda").fill_(255)
    ra.ra_layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, workspace=ws)
    return dx, dw, db


def check_backward(ra, dy, x, w, mean, rstd, dx=None):
    rows, cols = x.shape
    dx, dw, db = backward(ra, dy, x, w, mean, rstd, dx)
    dy64, r = dy.double(), rstd.double()[:, None]
    h, a = (x.double() - mean.double()[:, None]) * r, dy64 * w.double()
    c1, c2 = a.mean(1, keepdim=True), (a * h).mean(1, keepdim=True)
    want = r * (a - c1 - h * c2)
    k = (cols / 32 + 32) * U
    tol = r * k * (a.abs() + a.abs().mean(1, keepdim=True) + 2.01 * h.abs() * (a * h).abs().mean(1, keepdim=True))
    within(dx, want, ROUND[dx.dtype] * want.abs() + STEP[dx.dtype] + 1.01 * tol, "dx")
    for got, term, name in ((dw, dy64 * h, "dw"), (db, dy64, "db")):
        within(got, term.sum(0), 1.01 * (rows + 12) * U * term.abs().sum(0), name)


# columns of every way through the backward pass: 8, 16, 24, 32 a thread, on the 16-byte grid and off it, rows
# shared by 2 and 4 CTAs, and rows of any length
COLUMNS = [200, 203, 1024, 1537, 5120, 6001, 14000, 14001, 20000, 17001, 32768, 40000, 50001]


@pytest.mark.gpu
@pytest.mark.parametrize("cols", COLUMNS)
@pytest.mark.parametrize("dtype,value", [(F16, 1500.0), (F16, 60000.0), (BF16, 1504.0), (F32, 12345.678)])
def test_constant_rows_have_no_deviation(ra, dtype, value, cols):
    # xhat is 0, so the weight's gradient is too, whatever dy; dx is dy w less its mean
    gpu()
    gen = torch.Generator(device="cuda").manual_seed(cols)
    rows = 9
    x = torch.full((rows, cols), value, device="cuda").to(dtype)
    dy = torch.randn(rows, cols, generator=gen, device="cuda").to(dtype)
    w = torch.randn(cols, generator=gen, device="cuda") * 0.3 + 1
    mean, rstd = x[:, 0].float().contiguous(), torch.full((rows,), CONST_RSTD, device="cuda")
    _, dw, _ = backward(ra, dy, x, w, mean, rstd)
    assert (dw == 0).all(), float(dw.abs().max())
    if dtype is not F16:  # 316 times dy leaves fp16
        check_backward(ra, dy, x, w, mean, rstd)


@pytest.mark.gpu
@pytest.mark.parametrize("cols", COLUMNS)
@pytest.mark.parametrize("offset,std", [(1000.0, 1.0), (-1000.0, 0.1), (3.0, 1.0)])
def test_backward_far_from_zero(ra, cols, offset, std):
    gpu()
    gen = torch.Generator(device="cuda").manual_seed(cols + 1)
    rows = 40
    x = torch.randn(rows, cols, generator=gen, device="cuda") * std + offset
    dy = torch.randn(rows, cols, generator=gen, device="cuda") * 0.1
    w = torch.randn(cols, generator=gen, device="cuda") * 0.3 + 1
    mean = x.double().mean(1).float()
    rstd = ((x.double() - mean.double()[:, None]).square().mean(1) + EPS).rsqrt().float()
    check_backward(ra, dy, x, w, mean, rstd)


# rows and columns of every way through the forward pass, at few rows and at many
FORWARD = [(5, 64), (5, 300), (5, 768), (5000, 768), (5, 1000), (5000, 1003), (5, 1537), (5000, 701), (5000, 4095), (5, 5000), (5, 8191),
           (5, 9001), (5, 12288), (5, 14001), (5, 16384), (5, 20000), (5, 20001), (5, 32768), (3, 33001), (3, 70001)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", FORWARD)
@pytest.mark.parametrize("dtype,value", [(F32, 12345.678), (F32, 0.1), (F32, -1999.37), (F32, 10000001.0), (F32, 1e30), (F16, 2047.0),
                                         (F16, 0.33325), (BF16, 255.0)])
def test_a_constant_row_is_its_own_mean(ra, dtype, value, rows, cols):
    # its mean is the value to the last bit, so y is the bias and 1 / deviation 1 / sqrt(eps)
    gpu()
    for step in (0, 1):  # x and y in step, and one element apart
        x = torch.full((rows, cols), value, device="cuda").to(dtype)
        y = torch.empty(rows * cols + 1, device="cuda", dtype=dtype)[step:rows * cols + step].view(rows, cols)
        b = torch.randn(cols, device="cuda").to(dtype)
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        ra.ra_layernorm_forward(x, None, b, y, mean, rstd)
        assert torch.equal(mean, x[:, 0].float()), float((mean - x[:, 0].float()).abs().max())
        assert torch.equal(y, b.expand_as(y))
        assert ((rstd.double() - CONST_RSTD).abs() <= 4 * U * CONST_RSTD).all()


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [64, 1000, 1537, 9001, 16384, 33001])
@pytest.mark.parametrize("dtype", [F32, F16])
def test_rows_that_are_not_finite_keep_their_mean(ra, dtype, cols):
    gpu()
    x = torch.zeros(3, cols, device="cuda", dtype=dtype)
    x[0, 3], x[1, 5], x[2, 7] = float("inf"), -float("inf"), float("nan")
    y, mean, rstd = torch.empty_like(x), torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    ra.ra_layernorm_forward(x, None, None, y, mean, rstd)
    assert float(mean[0]) == float("inf") and float(mean[1]) == -float("inf") and bool(torch.isnan(mean[2]))
    assert bool(torch.isnan(y).all())


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [64, 1000, 1003, 1024, 1537, 6000, 20000, 33001])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_column_slices_of_one_matrix(ra, dtype, cols):
    # x, y, dy and dx side by side in one buffer: their address ranges overlap, their elements do not
    gpu()
    rows = 21
    gen = torch.Generator().manual_seed(cols)
    for gap in (0, 3, 8):
        both = torch.full((rows, 2 * cols + 2 * gap), 7.0, dtype=dtype, device="cuda")
        left, right = both[:, gap:gap + cols], both[:, cols + 2 * gap:]
        left.copy_(torch.randn(rows, cols, generator=gen))
        w, b = torch.randn(cols, generator=gen).cuda(), torch.randn(cols, generator=gen).cuda()
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        x = left.clone()
        test_layernorm.check_forward(ra, left, w, b, right, mean, rstd)
        assert torch.equal(left, x)
        right.copy_(torch.randn(rows, cols, generator=gen))
        dy = right.clone()
        other = torch.full((rows, 2 * cols + 2 * gap), 7.0, dtype=dtype, device="cuda")
        dx = other[:, cols + 2 * gap:]
        other[:, gap:gap + cols].copy_(dy)
        dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        test_layernorm.check_backward(ra, other[:, gap:gap + cols], left, w, mean, rstd, dx, dw, db)
        assert torch.equal(other[:, gap:gap + cols], dy) and torch.equal(left, x)
        for buffer in (both, other):  # and the gaps are left alone
            assert (buffer[:, :gap] == 7).all() and (buffer[:, gap + cols:cols + 2 * gap] == 7).all()


# Fake addresses that are never dereferenced: every case is refused on the host.
BASE = 0x7F0000000000
MB = 1 << 20


def test_slices_that_share_columns_are_refused(ra):
    def forward(y, ys, xs=200):
        return ra.lib().ra_layernorm_forward(BASE, xs, None, None, y, ys, None, None, 16, 64, 1e-5, 2, 2, None)

    def backward(dx, dxs, dys=200):
        return ra.lib().ra_layernorm_backward(BASE, dys, BASE + 4 * MB, 64, None, BASE + 5 * MB, BASE + 6 * MB, dx, dxs, None, None, 0, 16,
                                              64, 2, 2, None, 0, None)

    for call in (forward, backward):
        for apart in (2, 126, 274, 398, 402, 526):  # columns 1, 63, 137, 199 of 200, and the same a row later
            assert call(BASE + apart, 200) == ra.RA_ERR_ALIAS
        assert call(BASE - 126, 200) == call(BASE - 274, 200) == ra.RA_ERR_ALIAS
        assert call(BASE + 128, 199) == call(BASE + 128, 201) == ra.RA_ERR_ALIAS  # another stride
    # vectors between a matrix's rows
    assert ra.lib().ra_layernorm_forward(BASE, 200, BASE + 2 * MB, None, BASE + 4 * MB, 200, BASE + 128, None, 16, 64, 1e-5, 2, 0,
                                         None) == ra.RA_ERR_ALIAS


def strided(rows, cols, dtype, pad, shift, values=None):
    """A [rows, cols] view with `pad` elements between its rows, `shift` elements past an allocation's start."""
    base = torch.full((rows * (cols + pad) + shift,), 7.0, dtype=dtype, device="cuda")
    view = base[shift:].as_strided((rows, cols), (cols + pad, 1))
    if values is not None:
        view.copy_(values)
    return view


def assert_gaps_untouched(view):
    rows, cols = view.shape
    stride, start = view.stride(0), view.storage_offset()
    assert (view.as_strided((start,), (1,), 0) == 7).all()
    if rows > 1 and stride > cols:
        assert (view.as_strided((rows - 1, stride - cols), (stride, 1), start + cols) == 7).all()


# enough rows that every CTA, group of threads and place in shared memory comes to a second row, for each number of
# columns a thread, on the 16-byte grid and off it, and rows shared by several CTAs
MANY = [(20003, 200), (20003, 203), (6001, 501), (8001, 1024), (8001, 1003), (5001, 1536), (5001, 4095), (2501, 6000), (1001, 9001),
        (501, 12001), (501, 14000), (501, 14001), (701, 20000), (401, 20001), (501, 32768)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", MANY)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("pads,shift", [((0, 0, 0), 0), ((16, 48, 32), 0), ((48, 0, 16), 3)])
def test_every_row_and_stride(ra, dtype, rows, cols, pads, shift):
    # the matrices are in step (a pad is whole 16-byte lines) and have a stride each
    gpu()
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    x = strided(rows, cols, dtype, pads[0], shift, normal(rows, cols) * 2 + 0.7)
    y = strided(rows, cols, dtype, pads[1], shift)
    w, b = normal(cols) * 0.3 + 1, normal(cols) * 0.3
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ra.ra_layernorm_forward(x, w, b, y, mean, rstd)
    x64 = x.double()
    m = x64.mean(1, keepdim=True)
    r = ((x64 - m).square().mean(1, keepdim=True) + EPS).rsqrt()
    h = (x64 - m) * r
    k, top = (cols / 32 + 32) * U, x64.abs().amax(1, keepdim=True)
    want = h * w.double() + b.double()
    tol = w.double().abs() * k * (3 * h.abs() + 3 * top * r) + 2 * U * want.abs()
    within(y, want, ROUND[dtype] * want.abs() + STEP[dtype] + 1.01 * tol, "y")
    within(mean, m[:, 0], k * top[:, 0] + U * m[:, 0].abs(), "mean")
    within(rstd, r[:, 0], r[:, 0] * k * (3 + 3 * (top * r)[:, 0]), "rstd")
    assert_gaps_untouched(y)
    del x64, h, want, tol, y
    dy = strided(rows, cols, dtype, pads[2], shift, normal(rows, cols) * 0.1)
    dx = strided(rows, cols, dtype, pads[1], shift)
    check_backward(ra, dy, x, w, mean, rstd, dx)
    assert_gaps_untouched(dx)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(40, 6001), (700, 1537), (40, 20000), (40, 17001), (5, 60000)])
def test_in_a_graph(ra, rows, cols):
    # kernels with raised shared-memory limits, clusters, and several launches
    gpu()
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x, dy = (torch.randn(rows, cols, generator=gen, device="cuda").to(BF16) for _ in range(2))
    w = torch.randn(cols, generator=gen, device="cuda")
    ws = torch.empty(ra.ra_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")

    def outputs():
        return [torch.zeros_like(x), torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda"), torch.zeros_like(x),
                torch.zeros_like(w), torch.zeros_like(w)]

    def both(o):
        ra.ra_layernorm_forward(x, w, w, o[0], o[1], o[2])
        ra.ra_layernorm_backward(dy, x, w, o[1], o[2], o[3], o[4], o[5], workspace=ws)

    want, got = outputs(), outputs()
    both(want)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        both(got)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
