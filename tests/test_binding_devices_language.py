"""The binding of the embedding and the cross entropy refuses tensors of several devices, and of a device that is not
current, before the library is called. Tensors, devices and library are stand-ins: nothing is launched."""

import pytest
import torch

from test_binding_devices import OnDevice, library  # noqa: F401
from ring_all_reduce_02_gb300 import ra

BF16, F32, I64 = torch.bfloat16, torch.float32, torch.int64


def lookup(at, stream=None):
    ra.ra_embedding_forward(OnDevice(at("table"), 9, 8), OnDevice(at("tokens"), 4, dtype=I64), OnDevice(at("out"), 4, 8), stream=stream)


def lookup_gradient(at, stream=None):
    ra.ra_embedding_backward(OnDevice(at("dy"), 4, 8), OnDevice(at("tokens"), 4, dtype=I64), OnDevice(at("dtable"), 9, 8),
                             workspace=OnDevice(at("workspace"), 64), stream=stream)


def loss(at, stream=None):
    ra.ra_cross_entropy_forward(OnDevice(at("hidden"), 4, 8, dtype=BF16), OnDevice(at("weight"), 9, 8, dtype=BF16),
                                OnDevice(at("targets"), 4, dtype=I64), OnDevice(at("loss"), 4), OnDevice(at("lse"), 4),
                                workspace=OnDevice(at("workspace"), 64), stream=stream)


def loss_gradient(at, stream=None):
    ra.ra_cross_entropy_backward(OnDevice(at("hidden"), 4, 8, dtype=BF16), OnDevice(at("weight"), 9, 8, dtype=BF16),
                                 OnDevice(at("targets"), 4, dtype=I64), OnDevice(at("lse"), 4), OnDevice(at("dloss"), 4),
                                 OnDevice(at("dhidden"), 4, 8, dtype=BF16), OnDevice(at("dweight"), 9, 8, dtype=F32),
                                 workspace=OnDevice(at("workspace"), 64), stream=stream)


CALLS = {lookup: ("table", "tokens", "out"), lookup_gradient: ("dy", "tokens", "dtable", "workspace"),
         loss: ("hidden", "weight", "targets", "loss", "lse", "workspace"),
         loss_gradient: ("hidden", "weight", "targets", "lse", "dloss", "dhidden", "dweight", "workspace")}


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_on_the_current_device(library, call):  # noqa: F811
    for device in (0, 1):
        library.current = device
        call(lambda name: device)
        assert [stream for _, stream in library.calls] == [100 + device]
        library.calls.clear()


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_another_device_than_the_current_one(library, call):  # noqa: F811
    for current, device in ((0, 1), (1, 0)):
        library.current = current
        for stream in (None, 7):
            with pytest.raises(ValueError, match="current"):
                call(lambda name: device, stream=stream)
    assert not library.calls


@pytest.mark.parametrize("call,name", [(f, n) for f, names in CALLS.items() for n in names], ids=lambda v: getattr(v, "__name__", v))
def test_one_tensor_on_another_device(library, call, name):  # noqa: F811
    for device in (0, 1):
        library.current = device
        with pytest.raises(ValueError):
            call(lambda n: 1 - device if n == name else device)
    assert not library.calls


def test_types_and_missing_tensors(library):  # noqa: F811
    h, w, t = OnDevice(0, 4, 8, dtype=BF16), OnDevice(0, 9, 8, dtype=BF16), OnDevice(0, 4, dtype=I64)
    f, ws = OnDevice(0, 4), OnDevice(0, 64)
    with pytest.raises(TypeError, match="int32 or int64"):
        ra.ra_cross_entropy_forward(h, w, OnDevice(0, 4), f, f, workspace=ws)
    with pytest.raises(TypeError, match="int32 or int64"):
        ra.ra_embedding_forward(w, OnDevice(0, 4), h)
    with pytest.raises(TypeError, match="unsupported"):
        ra.ra_embedding_forward(OnDevice(0, 9, 8, dtype=torch.int32), t, OnDevice(0, 4, 8, dtype=torch.int32))
    with pytest.raises(ValueError, match="workspace"):
        ra.ra_cross_entropy_forward(h, w, t, f, f)
    with pytest.raises(ValueError, match="lse"):
        ra.ra_cross_entropy_backward(h, w, t, None, f, h, w, workspace=ws)
    with pytest.raises(ValueError, match="workspace"):
        ra.ra_embedding_backward(h, t, w)
    with pytest.raises(ValueError, match="dweight"):
        ra.ra_cross_entropy_backward(h, w, t, f, f, h, h, workspace=ws)
    with pytest.raises(ValueError, match="weight"):
        ra.ra_cross_entropy_forward(h, OnDevice(0, 9, 7, dtype=BF16), t, f, f, workspace=ws)
    assert not library.calls
