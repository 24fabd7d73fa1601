"""CPU checks of the decode-side operators' C boundary: the library exports what
include/ep_gb300_moe.h declares, the header is plain C, and every argument that
cannot be served is refused on the host with a message, before any launch."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import __graft_entry__
import combine_ep_layout_gb300 as ep
from combine_ep_layout_gb300 import _moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ep_gb300_moe.h")


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def test_exports_every_declared_symbol():
    with open(HEADER) as f:
        names = re.findall(r"^(?:int|void) (ep_\w+)\(", f.read(), flags=re.M)
    assert sorted(names) == ["ep_moe_create", "ep_moe_forward", "ep_moe_free", "ep_moe_layer", "ep_moe_status",
                             "ep_route", "ep_route_backward", "ep_w4_linear"]
    out = subprocess.run(["nm", "-D", "--defined-only", ep._native.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert set(names) <= exported


def test_header_is_plain_c_and_matches_the_binding():
    tu = '#include <stdio.h>\n#include "ep_gb300_moe.h"\nint main(void) { printf("%d %d %d %d", ' \
         "(int)sizeof(ep_route_cfg_t), (int)sizeof(ep_moe_cfg_t), (int)sizeof(ep_moe_weights_t), EP_FEW_TOKENS); " \
         "return 0; }\n"
    exe = os.path.join(ROOT, "combine_ep_layout_gb300", "_build", "moe_abi_sizes")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-x", "c", "-",
                    "-o", exe], input=tu, text=True, check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(ep.ep_route_cfg_t), ctypes.sizeof(ep.ep_moe_cfg_t),
                   ctypes.sizeof(ep.ep_moe_weights_t), ep.EP_FEW_TOKENS]


P = 0x1000           # an aligned address that nothing dereferences


def route(L, cfg, logits=P, dtype=ep.EP_FP32, stride=64, bias=None, n=1, idx=P, w=P):
    return L.ep_route(ctypes.byref(cfg) if cfg else None, logits, dtype, stride, bias, n, idx, w, None)


@pytest.mark.parametrize("bad", [dict(num_experts=0), dict(num_experts=2049), dict(topk=0), dict(topk=17),
                                 dict(topk=9, num_experts=8), dict(score=2), dict(renormalize=2),
                                 dict(scale=float("inf")), dict(scale=float("nan"))])
def test_route_cfg_is_checked(bad):
    L = _moe._load()
    cfg = ep.ep_route_cfg_t(**{**dict(num_experts=64, topk=8, score=0, renormalize=1, scale=1.0), **bad})
    assert route(L, cfg, n=0, stride=4096) == ep.EP_EINVAL and ep.ep_last_error()


@pytest.mark.parametrize("bad", [dict(logits=None), dict(logits=P + 2), dict(dtype=ep.EP_FP8_E4M3),
                                 dict(stride=63), dict(n=-1), dict(n=(1 << 24) + 1), dict(idx=None), dict(w=None),
                                 dict(idx=P + 4), dict(w=P + 2), dict(bias=P + 1),
                                 dict(dtype=ep.EP_BF16, logits=P + 1)])
def test_route_arguments_are_checked(bad):
    L = _moe._load()
    assert route(L, ep.make_route_cfg(64, 8), **bad) == ep.EP_EINVAL and ep.ep_last_error()


def test_route_null_cfg_and_empty_batches():
    L = _moe._load()
    assert route(L, None) == ep.EP_EINVAL
    assert route(L, ep.make_route_cfg(64, 8), logits=None, n=0, idx=None, w=None) == ep.EP_OK


@pytest.mark.parametrize("bad", [dict(logits=None), dict(idx=None), dict(g=None), dict(d=None), dict(d=P + 2),
                                 dict(g=P + 2), dict(idx=P + 4), dict(ds=63), dict(stride=63), dict(n=-1)])
def test_route_backward_arguments_are_checked(bad):
    L = _moe._load()
    a = {**dict(logits=P, stride=64, idx=P, g=P, n=1, d=P, ds=64), **bad}
    assert L.ep_route_backward(ctypes.byref(ep.make_route_cfg(64, 8)), a["logits"], ep.EP_FP32, a["stride"], a["idx"],
                               a["g"], a["n"], a["d"], a["ds"], None) == ep.EP_EINVAL
    assert ep.ep_last_error()


@pytest.mark.parametrize("bad", [dict(n=-1), dict(n=65), dict(rows=0), dict(rows=(1 << 24) + 1), dict(cols=0),
                                 dict(cols=100), dict(cols=1 << 19), dict(group=16), dict(group=256),
                                 dict(group=128, cols=192), dict(x=None), dict(q=None), dict(s=None), dict(out=None),
                                 dict(x=P + 8), dict(q=P + 8), dict(s=P + 2), dict(out=P + 2), dict(dtype=2)])
def test_w4_arguments_are_checked(bad):
    L = _moe._load()
    a = {**dict(x=P, n=1, q=P, s=P, rows=16, cols=256, group=64, out=P, dtype=ep.EP_FP32), **bad}
    assert L.ep_w4_linear(a["x"], a["n"], a["q"], a["s"], a["rows"], a["cols"], a["group"], a["out"], a["dtype"],
                          None) == ep.EP_EINVAL
    assert ep.ep_last_error()


def test_w4_of_no_tokens_launches_nothing():
    assert _moe._load().ep_w4_linear(None, 0, None, None, 16, 256, 64, None, ep.EP_FP32, None) == ep.EP_OK


@pytest.mark.parametrize("bad", [dict(hidden_dim=0), dict(hidden_dim=12), dict(hidden_dim=32776),
                                 dict(intermediate_dim=4), dict(intermediate_dim=100), dict(num_experts=0),
                                 dict(num_experts=2049), dict(num_expert_per_token=0), dict(num_expert_per_token=17),
                                 dict(max_tokens=0), dict(max_tokens=65), dict(weight_dtype=1),
                                 dict(group_size=32), dict(weight_dtype=4, group_size=0),
                                 dict(weight_dtype=4, group_size=48), dict(activation=2),
                                 dict(weight_dtype=4, group_size=128, hidden_dim=192)])
def test_moe_cfg_is_checked(bad):
    L = _moe._load()
    base = dict(hidden_dim=256, intermediate_dim=128, num_experts=8, num_expert_per_token=2, max_tokens=4,
                weight_dtype=0, group_size=0, activation=0)
    m = ctypes.c_void_p(1)
    assert L.ep_moe_create(ctypes.byref(ep.ep_moe_cfg_t(**{**base, **bad})), ctypes.byref(m)) == ep.EP_EINVAL
    assert m.value is None and ep.ep_last_error()


def test_moe_null_arguments():
    L = _moe._load()
    assert L.ep_moe_create(None, None) == ep.EP_EINVAL
    assert L.ep_moe_forward(None, P, 1, P, P, None, None, P, 0, None) == ep.EP_EINVAL
    rc = ep.make_route_cfg(8, 2)
    assert L.ep_moe_layer(None, ctypes.byref(rc), P, 1, P, ep.EP_FP32, 8, None, None, None, P, P, P, 0,
                          None) == ep.EP_EINVAL
    assert L.ep_moe_status(None, None) == ep.EP_EINVAL
    L.ep_moe_free(None)


def test_the_binding_refuses_what_is_not_on_the_gpu():
    rc = ep.make_route_cfg(8, 2)
    z, i, w = torch.zeros(3, 8), torch.zeros((3, 2), dtype=torch.int64), torch.zeros(3, 2)
    with pytest.raises(ValueError, match="CUDA"):
        ep.ep_route(rc, z, i, w)
    with pytest.raises(ValueError, match="CUDA"):
        ep.ep_route_backward(rc, z, i, w, z)
    with pytest.raises(ValueError, match="CUDA"):
        ep.ep_w4_linear(torch.zeros(1, 64, dtype=torch.bfloat16), torch.zeros((4, 32), dtype=torch.uint8),
                        torch.zeros(4, 1), torch.zeros(1, 4))
    with pytest.raises(ValueError, match="CUDA"):
        ep.EpMoeWeights(torch.zeros((2, 16, 8), dtype=torch.bfloat16), torch.zeros((2, 8, 8), dtype=torch.bfloat16))


@pytest.mark.gpu
def test_handle_refusals_on_the_gpu():
    L = _moe._load()
    cfg = ep.make_moe_cfg(64, 32, 8, 2, max_tokens=4)
    m = ep.EpMoe(cfg)
    w = ep.EpMoeWeights(torch.zeros((8, 64, 64), dtype=torch.bfloat16, device="cuda"),
                        torch.zeros((8, 64, 32), dtype=torch.bfloat16, device="cuda"))
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros((4, 2), dtype=torch.int64, device="cuda")
    tw = torch.zeros((4, 2), device="cuda")
    out = torch.empty_like(x)

    def call(n=4, x=x.data_ptr(), i=idx.data_ptr(), t=tw.data_ptr(), wt=w.c, bias=None, o=out.data_ptr(), dt=0):
        return L.ep_moe_forward(m.ptr, x, n, i, t, wt, bias, o, dt, None)
    assert call() == ep.EP_OK
    assert call(n=0, x=None, i=None, t=None, wt=None, o=None) == ep.EP_OK
    for bad in (dict(n=-1), dict(n=5), dict(x=None), dict(i=None), dict(t=None), dict(wt=None), dict(o=None),
                dict(x=x.data_ptr() + 2), dict(o=out.data_ptr() + 8), dict(bias=out.data_ptr() + 2),
                dict(i=idx.data_ptr() + 4), dict(t=tw.data_ptr() + 2), dict(dt=2),
                dict(wt=ep.ep_moe_weights_t(w.c.w13, tw.data_ptr(), w.c.w2, tw.data_ptr())),
                dict(wt=ep.ep_moe_weights_t(None, None, w.c.w2, None)),
                dict(wt=ep.ep_moe_weights_t(w.c.w13 + 2, None, w.c.w2, None))):
        assert call(**bad) == ep.EP_EINVAL, bad
        assert ep.ep_last_error()
    # a router of another shape than the handle's
    z = torch.zeros((4, 8), device="cuda")
    with pytest.raises(ep.EpError, match="handle's"):
        m.layer(ep.make_route_cfg(8, 1), x, z, w, idx, tw, out)
    with pytest.raises(ValueError, match="expected"):
        ep.EpMoe(ep.make_moe_cfg(64, 40, 8, 2)).forward(x, idx, tw, w, out)
    with pytest.raises(ValueError, match="weight_dtype"):
        ep.EpMoe(ep.make_moe_cfg(64, 32, 8, 2, 4, "int4", 32)).forward(x, idx, tw, w, out)
    with pytest.raises(ValueError, match="contiguous"):
        m.forward(x.t().contiguous().t(), idx, tw, w, out)
    m.free()
    with pytest.raises(ep.EpError, match="freed"):
        m.forward(x, idx, tw, w, out)
