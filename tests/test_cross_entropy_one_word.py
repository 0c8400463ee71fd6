"""A head of one word, cut out of a wider matrix: the distance to a next row, which there is not, decides nothing."""

import pytest
import torch

from test_binding_devices import OnDevice
from test_cross_entropy import BF16, F16, F32, I64, check_backward, check_forward, generator, gpu, ra  # noqa: F401


class Recorder:
    """Stands in for the library: what it is called with."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.mark.parametrize("stride", [9, 10, 16, 64])
@pytest.mark.parametrize("cols", [8, 9, 16])
def test_workspace_is_for_the_stride_that_the_calls_pass(monkeypatch, cols, stride):
    from ring_all_reduce_02_gb300 import ra as binding

    fake = Recorder()
    binding._Torch.load()
    monkeypatch.setattr(binding, "_lib", fake)
    monkeypatch.setattr(binding._Torch, "current_device", lambda: 0, raising=False)
    monkeypatch.setattr(binding._Torch, "current_stream", lambda device: 0)

    def on_device(*shape, dtype=F32, strides=None):
        t = OnDevice(0, *shape, dtype=dtype)
        if strides:
            t.t = torch.zeros(256, dtype=dtype).as_strided(shape, strides)
        return t

    for words in (1, 2):
        if words > 1 and stride < cols:
            continue
        h, w = on_device(3, cols, dtype=BF16), on_device(words, cols, dtype=BF16, strides=(stride, 1))
        f = on_device(3)
        fake.calls.clear()
        binding.ra_cross_entropy_workspace(h, w)
        binding.ra_cross_entropy_forward(h, w, on_device(3, dtype=I64), f, f, workspace=f)
        binding.ra_cross_entropy_backward(h, w, on_device(3, dtype=I64), f, f, h, w, workspace=f)
        (_, asked), (_, forward), (_, backward) = fake.calls
        assert asked[:2] == forward[2:4] == backward[2:4]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("cols,stride", [(9, 16), (9, 9), (9, 10), (16, 17), (16, 24), (72, 73), (73, 80)])
def test_one_word(ra, dtype, cols, stride):  # noqa: F811
    gpu()
    gen = generator(cols + stride)
    rows = 5
    h = torch.randn(rows, cols, generator=gen, device="cuda").to(dtype)
    w = torch.randn(2, stride, generator=gen, device="cuda").to(dtype)[:1, :cols]
    targets = torch.zeros(rows, dtype=I64, device="cuda")
    lse = check_forward(ra, h, w, targets)
    check_backward(ra, h, w, targets, lse, None, torch.empty_like(h), torch.zeros(2, stride, dtype=dtype, device="cuda")[:1, :cols])
