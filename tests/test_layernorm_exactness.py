"""What layer norm owes to rows that lie far from zero, and to every row of a call.

Tolerances as in test_layernorm.py, with u = 2^-24, but xhat = (x - mean) rstd
is held to its own two roundings (3 u |xhat|) wherever the row lies: no term in
|mean|. Everything is compared in 64 bits on the GPU."""

import pytest
import torch

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
COLUMNS = [200, 203, 1024, 1537, 5120, 6001, 14000, 14001, 20000, 17001, 32768, 40000]


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
