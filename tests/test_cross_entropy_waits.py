"""The bounded waits inside the cross entropy's kernels: where one gives up, the launch ends, every result says so, and the
next call is as any other."""

import pytest
import torch

from test_binding_devices import OnDevice
from test_cross_entropy import BF16, F16, I64, check_backward, check_forward, draw_targets, generator, gpu, matrix, ra  # noqa: F401

WITHHELD = {"tiles": 1, "operand": 2, "products": 3, "results": 4}
# one row, few and many, the weight in place and packed, one piece of the words and several. 512 columns and more: a pair takes
# no tile ahead of the one before the last. More than two tiles for each of the 76 pairs, or results that nobody reads stop no one
SIZES = [(1, 512, 50257), (200, 520, 45000), (700, 516, 20011), (300, 515, 30011), (9000, 512, 26000)]


def operands(rows, cols, vocab, dtype):
    gen = generator(rows + vocab)
    targets = draw_targets(rows, vocab, gen, I64, range(1, rows, 7))
    return matrix(rows, cols, dtype, gen), matrix(vocab, cols, dtype, gen, std=0.02), targets


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("withheld", WITHHELD)
@pytest.mark.parametrize("rows,cols,vocab", SIZES)
def test_waits_that_give_up(ra, rows, cols, vocab, withheld, dtype):  # noqa: F811
    gpu()
    h, w, targets = operands(rows, cols, vocab, dtype)
    counts = targets != -100
    loss, lse = torch.full((rows,), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda")
    ws = torch.zeros(ra.ra_cross_entropy_workspace(h, w), dtype=torch.uint8, device="cuda")
    ra.ra_selftest_cross_entropy_timeout(h, w, targets, loss, lse, withhold=WITHHELD[withheld], workspace=ws)
    torch.cuda.synchronize()
    assert torch.isnan(loss[counts]).all() and torch.isnan(lse[counts]).all()
    assert (loss[~counts] == 0).all() and (lse[~counts] == 0).all()
    ra.ra_cross_entropy_forward(h, w, targets, loss, lse, workspace=ws)  # the same workspace, and nothing is left of it
    again = check_forward(ra, h, w, targets)
    assert torch.equal(lse, again)

    ws = torch.zeros(ra.ra_cross_entropy_workspace(h, w, backward=True), dtype=torch.uint8, device="cuda")
    dh, dw = torch.full_like(h, 7.0), torch.full_like(w, 7.0)
    ra.ra_selftest_cross_entropy_timeout(h, w, targets, lse=lse, dhidden=dh, dweight=dw, withhold=WITHHELD[withheld], workspace=ws)
    torch.cuda.synchronize()
    assert torch.isnan(dh[counts]).all() and (dh[~counts] == 0).all() and torch.isnan(dw).all()
    ra.ra_cross_entropy_backward(h, w, targets, lse, None, dh, dw, workspace=ws)
    other_dh, other_dw = torch.empty_like(h), torch.empty_like(w)
    if rows < 1000:
        check_backward(ra, h, w, targets, lse, None, other_dh, other_dw)
        assert torch.equal(dh, other_dh) and torch.equal(dw, other_dw)
    assert torch.isfinite(dh).all() and torch.isfinite(dw).all()


# Fake addresses that are never dereferenced: every case is refused on the host.
BASE = 0x7F0000000000
MB = 1 << 20


def test_refusals(ra):  # noqa: F811
    need = ra.lib().ra_cross_entropy_workspace(BASE, 64, 16, 64, 100, 2, 1)

    def call(withhold=1, dt=2, h=BASE, dh=BASE + 8 * MB, dw=BASE + 10 * MB, n=need, cols=64):
        return ra.lib().ra_selftest_cross_entropy_timeout(h, BASE + 2 * MB, BASE + 4 * MB, BASE + 5 * MB, BASE + 6 * MB, dh, dw, 16, cols, 100, dt,
                                                          withhold, BASE + 16 * MB, n, None)

    bad = ra.RA_ERR_INVALID_ARG
    assert call(withhold=0) == call(withhold=5) == call(withhold=-1) == call(h=0) == call(n=need - 1) == call(cols=0) == bad
    assert call(dh=0, dw=0, h=0) == bad and call(dt=0) == ra.RA_ERR_UNSUPPORTED and call(dh=BASE) == ra.RA_ERR_ALIAS
    h = torch.zeros(4, 8, dtype=BF16)
    with pytest.raises(ValueError, match="CUDA"):
        ra.ra_selftest_cross_entropy_timeout(h, h, torch.zeros(4, dtype=I64), workspace=h)


def test_binding_refusals(monkeypatch):
    from ring_all_reduce_02_gb300 import ra as binding

    calls = []

    class Fake:
        def __getattr__(self, name):
            return lambda *args: calls.append(name) or 0

    binding._Torch.load()
    monkeypatch.setattr(binding, "_lib", Fake())
    monkeypatch.setattr(binding._Torch, "current_device", lambda: 0, raising=False)
    monkeypatch.setattr(binding._Torch, "current_stream", lambda device: 0)

    def call(h=(4, 8), w=(9, 8), t=4, tdtype=I64, n=4, dh=(4, 8), dw=(9, 8), wdtype=BF16, ws=64, device=0):
        def on(*shape, dtype=torch.float32, at=0):
            return OnDevice(at, *shape, dtype=dtype)

        binding.ra_selftest_cross_entropy_timeout(
            on(*h, dtype=BF16), on(*w, dtype=wdtype, at=device), on(t, dtype=tdtype), on(n), on(n), on(*dh, dtype=BF16), on(*dw, dtype=BF16),
            workspace=None if ws is None else on(ws))

    call()
    assert calls == ["ra_selftest_cross_entropy_timeout"]
    with pytest.raises(TypeError, match="int64"):
        call(tdtype=torch.int32)
    for wrong in (dict(h=(4,)), dict(w=(9, 7)), dict(t=3), dict(n=3), dict(dh=(3, 8)), dict(dw=(8, 8)), dict(wdtype=F16), dict(ws=None), dict(device=1)):
        with pytest.raises(ValueError):
            call(**wrong)
    assert len(calls) == 1
