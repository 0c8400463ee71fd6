"""Numbers that the C interface's 64 bits do not hold: the binding does not cut them off. Tensors and library are stand-ins."""

import pytest
import torch

from test_binding_devices import OnDevice
from ring_all_reduce_02_gb300 import ra

BF16, I64 = torch.bfloat16, torch.int64


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append(args) or 0


@pytest.fixture()
def library(monkeypatch):
    fake = Recorder()
    ra._Torch.load()
    monkeypatch.setattr(ra, "_lib", fake)
    monkeypatch.setattr(ra._Torch, "current_device", lambda: 0, raising=False)
    monkeypatch.setattr(ra._Torch, "current_stream", lambda device: 0)
    return fake


@pytest.mark.parametrize("padding,given", [(None, -1), (0, 0), (8, 8), (9, -1), (-1, -1), (-7, -1), (2 ** 31, -1), (2 ** 63, -1), (2 ** 64 + 5, -1),
                                           (-2 ** 64 + 5, -1)])
def test_a_padding_outside_the_vocabulary_is_none(library, padding, given):
    ra.ra_embedding_backward(OnDevice(0, 4, 8), OnDevice(0, 4, dtype=I64), OnDevice(0, 9, 8), padding=padding, workspace=OnDevice(0, 64))
    assert library.calls[0][4] == given


def test_ignore_has_64_bits(library):
    h, w, t, f = OnDevice(0, 4, 8, dtype=BF16), OnDevice(0, 9, 8, dtype=BF16), OnDevice(0, 4, dtype=I64), OnDevice(0, 4)
    calls = (lambda n: ra.ra_cross_entropy_forward(h, w, t, f, f, ignore=n, workspace=f),
             lambda n: ra.ra_cross_entropy_backward(h, w, t, f, f, h, w, ignore=n, workspace=f))
    for call in calls:
        for n in (-2 ** 63, -100, 0, 2 ** 63 - 1):
            call(n)
            assert library.calls.pop()[6] == n
        for n in (2 ** 63, -2 ** 63 - 1, 2 ** 64 - 100, 2 ** 64 + 5):
            with pytest.raises(ValueError, match="64 bits"):
                call(n)
            assert not library.calls
