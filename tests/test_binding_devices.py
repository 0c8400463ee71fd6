"""The training operators' binding refuses tensors of several devices, and of a device that is not current, before
the library is called. Tensors, devices and library are stand-ins: nothing is launched and no GPU is needed."""

import pytest
import torch

from ring_all_reduce_02_gb300 import ra

F32, F8 = torch.float32, torch.float8_e4m3fn


class OnDevice:
    """A host tensor that says it is on a CUDA device."""

    def __init__(self, device, *shape, dtype=F32):
        self.t, self.device_index = torch.zeros(*shape, dtype=dtype), device

    is_cuda = True

    def get_device(self):
        return self.device_index

    def __getattr__(self, name):
        return getattr(self.t, name)


class Library:
    """Records the calls, and their stream."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args[-1]))
            return 0

        return call


@pytest.fixture()
def library(monkeypatch):
    fake = Library()
    ra._Torch.load()
    monkeypatch.setattr(ra, "_lib", fake)
    monkeypatch.setattr(ra._Torch, "current_device", lambda: fake.current, raising=False)
    monkeypatch.setattr(ra._Torch, "current_stream", lambda device: 100 + device)
    fake.current = 0
    return fake


def forward(at, stream=None):
    ra.ra_layernorm_forward(OnDevice(at("x"), 4, 8), OnDevice(at("weight"), 8), OnDevice(at("bias"), 8), OnDevice(at("y"), 4, 8),
                            OnDevice(at("mean"), 4), OnDevice(at("rstd"), 4), stream=stream)


def backward(at, stream=None):
    ra.ra_layernorm_backward(OnDevice(at("dy"), 4, 8), OnDevice(at("x"), 4, 8), OnDevice(at("weight"), 8), OnDevice(at("mean"), 4),
                             OnDevice(at("rstd"), 4), OnDevice(at("dx"), 4, 8), OnDevice(at("dweight"), 8), OnDevice(at("dbias"), 8),
                             workspace=OnDevice(at("workspace"), 64), stream=stream)


def norm(at, stream=None):
    ra.ra_grad_norm([OnDevice(at("first"), 3), OnDevice(at("second"), 5)], 1.0, OnDevice(at("out"), 2), OnDevice(at("workspace"), 64),
                    stream=stream)


def adamw(at, stream=None):
    def two(name, dtype=F32):
        return [OnDevice(at(name), 3, dtype=dtype), OnDevice(at(name + " 2"), 5, dtype=dtype)]

    def scales(name):
        return [OnDevice(at(name), 1), OnDevice(at(name + " 2"), 1)]

    tensors = ra.adamw_tensors(two("param"), two("grad"), two("m", F8), two("v", F8), scales("m scale"), scales("v scale"), 0.0,
                               two("copy"))
    ra.ra_adamw(tensors, lr=1e-3, step=1, grad_scale=OnDevice(at("grad_scale"), 1), stream=stream)


CALLS = {forward: ("x", "weight", "bias", "y", "mean", "rstd"),
         backward: ("dy", "x", "weight", "mean", "rstd", "dx", "dweight", "dbias", "workspace"),
         norm: ("first", "second", "out", "workspace"),
         adamw: tuple(name + two for name in ("param", "grad", "m", "v", "m scale", "v scale", "copy") for two in ("", " 2"))
         + ("grad_scale",)}


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_on_the_current_device(library, call):
    for device in (0, 1):
        library.current = device
        call(lambda name: device)
        assert [stream for _, stream in library.calls] == [100 + device]
        library.calls.clear()


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_another_device_than_the_current_one(library, call):
    for current, device in ((0, 1), (1, 0)):
        library.current = current
        for stream in (None, 7):
            with pytest.raises(ValueError, match="current"):
                call(lambda name: device, stream=stream)
    assert not library.calls


@pytest.mark.parametrize("call,name", [(f, n) for f, names in CALLS.items() for n in names], ids=lambda v: getattr(v, "__name__", v))
def test_one_tensor_on_another_device(library, call, name):
    for device in (0, 1):
        library.current = device
        with pytest.raises(ValueError):
            call(lambda n: 1 - device if n == name else device)
    assert not library.calls


def test_no_gradients_at_all(library):
    ra.ra_grad_norm([], 1.0, OnDevice(0, 2), OnDevice(0, 64))
    assert library.calls == [("ra_grad_norm", 100)]
    with pytest.raises(ValueError):
        ra.ra_grad_norm([], 1.0, OnDevice(0, 2), OnDevice(1, 64))
    with pytest.raises(ValueError, match="current"):
        ra.ra_grad_norm([], 1.0, OnDevice(1, 2), OnDevice(1, 64))
    with pytest.raises(ValueError):
        ra.ra_grad_norm([], 1.0, torch.zeros(2), torch.zeros(64))


def test_a_missing_workspace_is_refused(library):
    with pytest.raises(ValueError, match="workspace"):
        ra.ra_grad_norm([OnDevice(0, 3)], 1.0, OnDevice(0, 2), None)
    with pytest.raises(ValueError, match="out"):
        ra.ra_grad_norm([OnDevice(0, 3)], 1.0, None, OnDevice(0, 64))
    assert not library.calls
