"""The router's gradient entry by entry, relative to each entry's own terms: sigmoid scores
far above zero, where f is near 1 and 1 - f has to keep its bits, and far below.

dz_k = w_k (g_k - sum g a) (1 - f_k) with w_k = f_k, or a_k where renormalised.  With |z| <= D
an exp is off by 2^-24 D + 2^-22, for D <= 80 by 5e-6; f and 1 - f have one each, a two and a
sum's rounding: below 2e-5 of w_k (|g_k| + sum |g a|) (1 - f_k); bf16 adds 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import combine_ep_layout_gb300 as ep

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("lo,hi", [(8, 30), (-5, 17), (40, 80), (-80, -20)])
@pytest.mark.parametrize("k", [1, 6, 12])
def test_each_entry_of_the_sigmoid_gradient(k, lo, hi, renorm, dtype):
    n, e, scale = 37, 64, 2.5
    gen = torch.Generator().manual_seed(k + hi)
    z = (torch.rand((n, e), generator=gen) * (hi - lo) + lo).to(dtype).cuda()
    g = torch.randn((n, k), generator=gen).cuda()
    cfg = ep.make_route_cfg(e, k, "sigmoid", renorm, scale)
    idx = torch.empty((n, k), dtype=torch.int64, device="cuda")
    w = torch.empty((n, k), device="cuda")
    ep.ep_route(cfg, z, idx, w)
    dz = torch.full_like(z, float("nan"))
    ep.ep_route_backward(cfg, z, idx, g, dz)
    zk = torch.gather(z, 1, idx).double().cpu().numpy()
    f, rest = 1.0 / (1.0 + np.exp(-zk)), 1.0 / (1.0 + np.exp(zk))
    gs = scale * g.double().cpu().numpy()
    if renorm:
        v = f / f.sum(1, keepdims=True)
        want, size = v * (gs - (gs * v).sum(1, keepdims=True)) * rest, \
            v * (np.abs(gs) + np.abs(gs * v).sum(1, keepdims=True)) * rest
    else:
        want, size = f * gs * rest, f * np.abs(gs) * rest
    got = torch.gather(dz, 1, idx).double().cpu().numpy()
    rel = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    assert (np.abs(got - want) <= 2e-5 * size + rel * np.abs(want) + 1e-37).all()
    assert (dz.scatter(1, idx, 0.0) == 0).all()
