"""CPU checks of the binding: tensors of different devices, tensors that are not on the
current device, and a stream of another device are refused before anything is launched."""
import pytest
import torch

import __graft_entry__
import combine_ep_layout_gb300 as ep
from combine_ep_layout_gb300 import _moe


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


class OnDevice:
    """What the binding asks of a CUDA tensor."""
    is_cuda = True

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device_index = torch.Size(shape), dtype, device

    def dim(self):
        return len(self.shape)

    def stride(self, d):
        n = 1
        for s in self.shape[d + 1:]:
            n *= s
        return n

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.device_index

    def data_ptr(self):
        return 0x1000


class Stream:
    def __init__(self, device):
        self.device_index, self.cuda_stream = device, 0


BF16, F32, I64, U8 = torch.bfloat16, torch.float32, torch.int64, torch.uint8
N, E, K = 3, 8, 2
CALLS = {
    "route": (lambda t, **k: ep.ep_route(ep.make_route_cfg(E, K), *t, **k),
              [((N, E), F32), ((N, K), I64), ((N, K), F32), ((E,), F32)]),
    "route_backward": (lambda t, **k: ep.ep_route_backward(ep.make_route_cfg(E, K), *t, **k),
                       [((N, E), F32), ((N, K), I64), ((N, K), F32), ((N, E), F32)]),
    "w4": (lambda t, **k: ep.ep_w4_linear(*t, **k),
           [((N, 64), BF16), ((16, 32), U8), ((16, 2), F32), ((N, 16), BF16)]),
}


@pytest.fixture
def no_launch(monkeypatch):
    def refuse(*a):
        raise AssertionError("launched")

    class Library:
        ep_route = ep_route_backward = ep_w4_linear = ep_moe_forward = ep_moe_layer = staticmethod(refuse)
    monkeypatch.setattr(_moe, "_load", lambda: Library)
    monkeypatch.setattr(_moe, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(_moe, "_current_device", lambda: 0, raising=False)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_one_device_and_the_current_one(name, no_launch):
    call, args = CALLS[name]
    with pytest.raises(AssertionError, match="launched"):
        call([OnDevice(*a, 0) for a in args])
    with pytest.raises(AssertionError, match="launched"):
        call([OnDevice(*a, 0) for a in args], stream=Stream(0))
    for other in range(len(args)):
        with pytest.raises(ValueError, match="device"):
            call([OnDevice(*a, int(i == other)) for i, a in enumerate(args)])
    with pytest.raises(ValueError, match="current device"):
        call([OnDevice(*a, 1) for a in args])
    with pytest.raises(ValueError, match="stream"):
        call([OnDevice(*a, 0) for a in args], stream=Stream(1))


def test_the_layer_takes_tensors_of_its_handles_device(no_launch):
    H, I = 16, 8
    m = ep.EpMoe.__new__(ep.EpMoe)
    m.cfg, m.device, m._m = ep.make_moe_cfg(H, I, E, K, N), 0, 1
    shapes = [((N, H), BF16), ((N, K), I64), ((N, K), F32), ((N, H), BF16), ((N, H), BF16), ((N, E), F32), ((E,), F32)]

    def call(devices, w_devices, layer):
        w = ep.EpMoeWeights(OnDevice((E, 2 * I, H), BF16, w_devices[0]), OnDevice((E, H, I), BF16, w_devices[1]))
        x, idx, tw, out, bias, z, sb = (OnDevice(*s, d) for s, d in zip(shapes, devices))
        if layer:
            m.layer(ep.make_route_cfg(E, K), x, z, w, idx, tw, out, bias=bias, select_bias=sb)
        else:
            m.forward(x, idx, tw, w, out, bias=bias)
    for layer in (False, True):
        with pytest.raises(AssertionError, match="launched"):
            call([0] * 7, (0, 0), layer)
        for w_devices in ((0, 1), (1, 0), (1, 1)):
            with pytest.raises(ValueError, match="device"):
                call([0] * 7, w_devices, layer)
        for other in range(7 if layer else 5):
            with pytest.raises(ValueError, match="device"):
                call([int(i == other) for i in range(7)], (0, 0), layer)
    m._m = None
