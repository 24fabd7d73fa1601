"""CPU checks of the boundary of the training losses and of the int8 path: the library
exports what the headers declare, the headers are plain C, and every argument that
cannot be served is refused on the host with a message, before any launch."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import __graft_entry__
import combine_ep_layout_gb300 as ep
from combine_ep_layout_gb300 import _balance, _i8
from test_moe_devices import OnDevice, Stream

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INCLUDE = os.path.join(ROOT, "include")
P = 0x1000           # an aligned address that nothing dereferences


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


@pytest.mark.parametrize("header,want", [
    ("ep_gb300_balance.h", ["ep_balance_backward", "ep_balance_create", "ep_balance_forward", "ep_balance_free"]),
    ("ep_gb300_i8.h", ["ep_i8_dispatch", "ep_i8_grouped", "ep_i8_linear", "ep_i8_quantize", "ep_i8_status"])])
def test_exports_every_declared_symbol(header, want):
    with open(os.path.join(INCLUDE, header)) as f:
        names = re.findall(r"^(?:int|void) (ep_\w+)\(", f.read(), flags=re.M)
    assert sorted(names) == want
    out = subprocess.run(["nm", "-D", "--defined-only", ep._native.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert set(names) <= {line.split()[-1] for line in out.splitlines() if " T " in line}


def test_headers_are_plain_c():
    tu = '#include <stdio.h>\n#include "ep_gb300_balance.h"\n#include "ep_gb300_i8.h"\nint main(void) { ' \
         'printf("%d %d", EP_ACT_NONE, EP_I8_MAX_COLS); return 0; }\n'
    exe = os.path.join(ROOT, "combine_ep_layout_gb300", "_build", "i8_abi_sizes")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", INCLUDE, "-x", "c", "-", "-o", exe], input=tu,
                   text=True, check=True)
    got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    assert got == "%d %d" % (ep.EP_ACT_NONE, ep.EP_I8_MAX_COLS)


@pytest.mark.parametrize("cfg,tokens,sequences", [
    (dict(num_experts=0), 8, 1), (dict(num_experts=2049), 8, 1), (dict(topk=17), 8, 1), (dict(score=2), 8, 1),
    (dict(renormalize=3), 8, 1), (dict(scale=float("nan")), 8, 1), ({}, 0, 1), ({}, (1 << 24) + 1, 1), ({}, 8, 0),
    ({}, 8, (1 << 20) + 1)])
def test_balance_configurations_are_checked(cfg, tokens, sequences):
    c = ep.ep_route_cfg_t(**{**dict(num_experts=64, topk=8, score=0, renormalize=1, scale=1.0), **cfg})
    b = ctypes.c_void_p(1)
    assert _balance._load().ep_balance_create(ctypes.byref(c), tokens, sequences, ctypes.byref(b)) == ep.EP_EINVAL
    assert ep.ep_last_error() and not b.value


def test_balance_null_handles():
    L = _balance._load()
    assert L.ep_balance_create(None, 1, 1, ctypes.byref(ctypes.c_void_p())) == ep.EP_EINVAL
    assert L.ep_balance_create(ctypes.byref(ep.make_route_cfg(8, 2)), 1, 1, None) == ep.EP_EINVAL
    assert L.ep_balance_forward(None, P, 1, 8, P, 1, None, 1, P, P, P, P, None) == ep.EP_EINVAL
    assert L.ep_balance_backward(None, P, 1, 8, P, 1, None, 1, P, P, P, P, 8, 0, None) == ep.EP_EINVAL
    L.ep_balance_free(None)


def quantize(x=P, dtype=ep.EP_BF16, stride=64, n=3, cols=64, q=P, scales=P):
    return _i8._load().ep_i8_quantize(None, x, dtype, stride, n, cols, q, scales, None)


@pytest.mark.parametrize("bad", [dict(x=None), dict(q=None), dict(scales=None), dict(x=P + 1), dict(dtype=ep.EP_FP32, x=P + 2),
                                 dict(q=P + 8), dict(scales=P + 2), dict(dtype=ep.EP_FP8_E4M3), dict(stride=63), dict(n=-1),
                                 dict(n=1 << 31), dict(cols=0), dict(cols=24), dict(cols=65552, stride=65552)])
def test_quantize_arguments_are_checked(bad):
    assert quantize(**bad) == ep.EP_EINVAL and ep.ep_last_error()


def test_empty_calls_launch_nothing():
    assert quantize(x=None, q=None, scales=None, n=0) == ep.EP_OK
    assert linear(x=None, xs=None, w=None, ws=None, out=None, n=0) == ep.EP_OK


def linear(x=P, xs=P, n=3, w=P, ws=P, rows=10, cols=64, act=ep.EP_ACT_NONE, out=P, dtype=ep.EP_BF16):
    return _i8._load().ep_i8_linear(x, xs, n, w, ws, rows, cols, act, out, dtype, None)


@pytest.mark.parametrize("bad", [dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(out=None), dict(x=P + 8), dict(w=P + 8),
                                 dict(xs=P + 2), dict(ws=P + 1), dict(out=P + 1), dict(dtype=ep.EP_FP32, out=P + 2),
                                 dict(dtype=ep.EP_FP8_E4M3), dict(n=-1), dict(n=(1 << 24) + 1), dict(rows=0),
                                 dict(rows=(1 << 24) + 1), dict(cols=0), dict(cols=40), dict(cols=1 << 17), dict(act=2),
                                 dict(act=-2), dict(act=0, rows=11)])
def test_linear_arguments_are_checked(bad):
    assert linear(**bad) == ep.EP_EINVAL and ep.ep_last_error()


def test_null_handles_and_status():
    L = _i8._load()
    assert L.ep_i8_dispatch(None, P, 0, P, P, None) == ep.EP_EINVAL
    assert L.ep_i8_grouped(None, P, P, P, P, 8, 16, -1, P, 0, None) == ep.EP_EINVAL
    assert L.ep_i8_status(None, None) == ep.EP_EINVAL


# ---------------------------------------------------- the binding's own checks

BF16, F32, I64, I32, I8 = torch.bfloat16, torch.float32, torch.int64, torch.int32, torch.int8
N, E, K, M = 3, 8, 2, 2


class Handle:
    """What the calls ask of an EpHandle."""
    def __init__(self, rows=N):
        self.cfg = ep.make_cfg(1, 64, N, E, K)
        self.device, self.recv_capacity, self.num_tokens, self._layout_of, self.ptr = 0, rows, N, None, None


def balance():
    b = ep.EpBalance.__new__(ep.EpBalance)
    b.cfg, b.device, b._b = ep.make_route_cfg(E, K), 0, None
    return b


CALLS = {
    "quantize": (lambda t, **k: ep.ep_i8_quantize(*t, **k), [((N, 64), BF16), ((N, 64), I8), ((N,), F32)]),
    "dispatch": (lambda t, **k: ep.ep_i8_dispatch(Handle(), *t, **k), [((N, 64), F32), ((N, 64), I8), ((N,), F32)]),
    "linear": (lambda t, **k: ep.ep_i8_linear(*t, **k),
               [((N, 64), I8), ((N,), F32), ((16, 64), I8), ((16,), F32), ((N, 16), BF16)]),
    "grouped": (lambda t, **k: ep.ep_i8_grouped(Handle(), *t, **k),
                [((N, 64), I8), ((N,), F32), ((E, 16, 64), I8), ((E, 16), F32), ((N, 16), BF16)]),
    "balance": (lambda t, **k: balance().forward(*t[:6], seq_offsets=t[6], **k),
                [((N, E), F32), ((N, K), I64), ((M, E), I32), ((M, E), F32), ((M + 1,), I32), ((2,), F32), ((M + 1,), I32)]),
    "balance_backward": (lambda t, **k: balance().backward(*t[:6], seq_offsets=t[6], **k),
                         [((N, E), BF16), ((N, K), I64), ((M, E), I32), ((M + 1,), I32), ((2,), F32), ((N, E), BF16),
                          ((M + 1,), I32)]),
}
ONE_OF_EACH = [(name, i) for name, (_, want) in CALLS.items() for i in range(len(want))]


@pytest.fixture
def no_launch(monkeypatch):
    class Nothing:
        def __getattr__(self, name):
            def call(*args):
                raise AssertionError("%s was called" % name)
            return call
    for m in (_i8, _balance):
        monkeypatch.setattr(m, "_load", lambda: Nothing())
    monkeypatch.setattr(_i8, "_current_device", lambda: 0)


@pytest.mark.parametrize("name,i", ONE_OF_EACH)
def test_a_tensor_of_another_device_type_or_shape_is_refused(no_launch, name, i):
    call, want = CALLS[name]
    with pytest.raises(ValueError):
        call([OnDevice(s, d, int(j == i)) for j, (s, d) in enumerate(want)])
    with pytest.raises(ValueError):
        call([OnDevice(s, torch.float64 if j == i else d, 0) for j, (s, d) in enumerate(want)])
    with pytest.raises(ValueError):
        call([OnDevice((*s[:-1], s[-1] + 1) if j == i else s, d, 0) for j, (s, d) in enumerate(want)])


@pytest.mark.parametrize("name", list(CALLS))
def test_streams_and_other_devices_are_refused(no_launch, name):
    call, want = CALLS[name]
    with pytest.raises(ValueError):
        call([OnDevice(s, d, 1) for s, d in want])
    with pytest.raises((ValueError, ep.EpError)):
        call([OnDevice(s, d, 0) for s, d in want], stream=Stream(1))


def test_activations_are_checked(no_launch):
    _, want = CALLS["linear"]
    with pytest.raises(ValueError):
        ep.ep_i8_linear(*[OnDevice(s, d, 0) for s, d in want], activation="relu")
    with pytest.raises(ValueError):          # a gated out has half the columns
        ep.ep_i8_linear(*[OnDevice(s, d, 0) for s, d in want], activation="silu")
