"""The router and its gradient against a plain implementation in 64 bits.

Ids have to be equal (ties go to the lower id).  Weights: with |z - peak| <= D
the argument of exp carries a rounding of 2^-24 D, exp itself 2 ulp, and a sum of
E terms in per-lane chains of E/32 and a 5-step tree (E/32 + 5) 2^-24; for D <= 40
and E <= 2048 that is below 1e-5 relative, which is the tolerance.  A gradient is
f (g - mean) with |f| <= 1: 2e-5 of the largest |g| of its row, and for bf16 the
rounding of 2^-8 relative.
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


def reference(z, k, score, renorm, scale, bias=None):
    """ids [n, k], weights, per-expert scores f and membership, in float64 numpy."""
    z = z.detach().double().cpu().numpy()
    n, e = z.shape
    live = z > -np.inf
    with np.errstate(all="ignore"):
        if score == "softmax":
            peak = np.where(live.any(1), np.where(live, z, -np.inf).max(1), 0.0)[:, None]
            x = np.where(live, np.where(z == peak, 1.0, np.exp(z - peak)), 0.0)
            s = x.sum(1, keepdims=True)
            f = np.where(s > 0, x / np.where(s > 0, s, 1.0), 0.0)
        else:
            f = np.where(live, 1.0 / (1.0 + np.exp(-z)), 0.0)
        key = z if bias is None else f + bias.double().cpu().numpy()[None]
    ids = np.full((n, k), -1, np.int64)
    w = np.zeros((n, k))
    member = np.zeros((n, e), bool)
    for t in range(n):
        order = sorted((j for j in range(e) if live[t, j] and key[t, j] > -np.inf),
                       key=lambda j: (-key[t, j], j))[:k]
        ids[t, :len(order)] = order
        v = f[t, order]
        if renorm and len(order):
            if score == "sigmoid":     # by the logarithms: all of them may underflow
                zz = z[t, order]
                v = np.where(zz < -40, zz, -np.log1p(np.exp(-np.maximum(zz, -40))))
                v = np.exp(v - v.max())
            v = v / v.sum()
        w[t, :len(order)] = scale * v
        member[t, order] = True
    return ids, w, f, member


def reference_grad(ids, w, f, member, g, score, renorm, scale):
    n, e = f.shape
    gw = np.zeros((n, e))
    a = np.zeros((n, e))
    for t in range(n):
        for k, j in enumerate(ids[t]):
            if j >= 0:
                gw[t, j] = g[t, k] * scale
                a[t, j] = w[t, k] / scale
    if renorm:
        d = a * (gw - (gw * a).sum(1, keepdims=True))
        return d * member * ((1 - f) if score == "sigmoid" else 1.0)
    if score == "softmax":
        return f * (gw - (gw * f).sum(1, keepdims=True))
    return gw * f * (1 - f)


def run(z, k, score, renorm, scale=1.0, bias=None):
    cfg = ep.make_route_cfg(z.shape[1], k, score, renorm, scale)
    idx = torch.full((z.shape[0], k), -77, dtype=torch.int64, device="cuda")
    w = torch.full((z.shape[0], k), float("nan"), device="cuda")
    ep.ep_route(cfg, z, idx, w, bias)
    return cfg, idx, w


def check(z, k, score, renorm, scale=1.0, bias=None, grad=True):
    cfg, idx, w = run(z, k, score, renorm, scale, bias)
    ids, ref, f, member = reference(z, k, score, renorm, scale, bias)
    assert np.array_equal(idx.cpu().numpy(), ids)
    np.testing.assert_allclose(w.cpu().numpy(), ref, rtol=1e-5, atol=1e-30)
    if not grad:
        return
    g = torch.randn(w.shape, generator=torch.Generator().manual_seed(3)).cuda()
    masked = idx < 0
    dz = torch.full_like(z, float("nan"))
    ep.ep_route_backward(cfg, z, idx, torch.where(masked, float("nan"), g), dz)
    want = reference_grad(ids, ref, f, member, g.double().cpu().numpy(), score, renorm, scale)
    far = np.abs(dz.double().cpu().numpy() - want)
    top = np.abs(g.cpu().numpy()).max(1, keepdims=True) * abs(scale)
    rel = 2.0 ** -8 if z.dtype == torch.bfloat16 else 0.0
    assert (far <= 2e-5 * top + rel * np.abs(want)).all()


def logits(n, e, dtype=torch.float32, seed=0, std=2.0):
    g = torch.Generator().manual_seed(1000 * e + n + seed)
    return (std * torch.randn((n, e), generator=g)).to(dtype).cuda()


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False),
                                          ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,e,k", [(1, 1, 1), (1, 64, 8), (3, 7, 7), (9, 32, 16), (17, 33, 2),
                                   (70, 60, 4), (33, 128, 6), (130, 250, 7), (64, 256, 8),
                                   (21, 257, 16), (5, 512, 8), (6, 1000, 1), (4, 2048, 16)])
def test_ids_weights_and_gradient(n, e, k, dtype, score, renorm):
    check(logits(n, e, dtype), k, score, renorm, scale=2.5 if score == "sigmoid" else 1.0)


def test_no_tokens():
    run(logits(0, 16), 4, "softmax", True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e", [8, 64, 256, 300])
def test_ties_go_to_the_lower_id(e, score):
    # few distinct values, both zeros among them, and rows of one value
    g = torch.Generator().manual_seed(e)
    z = torch.randint(-2, 3, (40, e), generator=g).float()
    z[3] = 0.0
    z[4] = -0.0
    z[5, ::2] = -0.0
    check(z.cuda(), 8, score, True)
    check(z.bfloat16().cuda(), 5, score, False)


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False),
                                          ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("mask", [float("-inf"), float("nan")])
def test_masked_scores(score, renorm, mask):
    z = logits(24, 96).clone()
    m = torch.rand((24, 96), generator=torch.Generator().manual_seed(5)).cuda() < 0.9
    z[m] = mask
    z[0] = mask                    # nothing left
    z[1] = mask
    z[1, 77] = -3.0                # one left
    z[2, :] = torch.finfo(torch.float32).min   # the type's lowest value is a score like any other
    z[2, 5] = mask
    check(z, 8, score, renorm)


@pytest.mark.parametrize("renorm", [True, False])
def test_sigmoid_scores_far_below_zero_keep_their_ratios(renorm):
    z = (logits(16, 64) - 30.0).clone()
    z[3] -= 70.0
    if renorm:
        z[4] -= 400.0              # every sigmoid underflows; the ratios do not
        z[4] = (z[4] * 64).round() / 64
    cfg, idx, w = run(z, 6, "sigmoid", renorm)
    ids, ref, f, member = reference(z[:4], 6, "sigmoid", renorm, 1.0)
    assert np.array_equal(idx[:4].cpu().numpy(), ids)
    np.testing.assert_allclose(w[:4].cpu().numpy(), ref, rtol=2e-5, atol=1e-37)
    if renorm:
        top = z[4].double().sort(descending=True).values[:6]
        torch.testing.assert_close(w[4].double(), torch.softmax(top, 0), rtol=2e-5, atol=0)


def test_infinite_scores():
    z = logits(4, 40).clone()
    z[0, 7] = float("inf")
    z[1, [3, 30]] = float("inf")
    check(z, 4, "softmax", True)
    check(z, 4, "softmax", False)
    check(z, 4, "sigmoid", False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_selection_bias(score, renorm):
    # biases a quarter apart, scores within a hundredth: the order is the biases'
    e = 48
    z = 0.01 * logits(20, e)
    b = 0.25 * torch.randperm(e, generator=torch.Generator().manual_seed(2)).float().cuda()
    z[4, 10:] = float("-inf")
    check(z, 6, score, renorm, bias=b, grad=False)
    b2 = b.clone()
    b2[::2] = float("-inf")        # never chosen
    b2[1] = float("nan")
    check(z, 6, score, renorm, bias=b2, grad=False)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_and_unaligned_rows(dtype):
    big = logits(40, 300, dtype)
    for view in (big[:, 1:257], big[::3, :256], big[5:, 44:], big[:, 3:35]):
        cfg, idx, w = run(view, 6, "softmax", False)
        cfg, idx2, w2 = run(view.contiguous(), 6, "softmax", False)
        assert torch.equal(idx, idx2) and torch.equal(w, w2)
        g = torch.randn_like(w)
        buf = torch.full((view.shape[0], view.shape[1] + 5), 9.0, dtype=dtype, device="cuda")
        d2 = torch.empty_like(view.contiguous())
        ep.ep_route_backward(cfg, view, idx, g, buf[:, 2:2 + view.shape[1]])
        ep.ep_route_backward(cfg, view.contiguous(), idx, g, d2)
        assert torch.equal(buf[:, 2:2 + view.shape[1]], d2)
        assert (buf[:, :2] == 9.0).all() and (buf[:, 2 + view.shape[1]:] == 9.0).all()


def test_skipped_ids_in_the_gradient():
    z = logits(4, 16)
    cfg, idx, w = run(z, 4, "softmax", True)
    g = torch.randn_like(w)
    idx[0] = -1
    idx[1, 2] = 99
    idx[2, 1] = -5
    d = torch.empty_like(z)
    ep.ep_route_backward(cfg, z, idx, g, d)
    assert (d[0] == 0).all() and torch.isfinite(d).all()
    keep = idx[1][[0, 1, 3]]
    p = torch.softmax(z[1][keep].double(), 0)
    gg = g[1][[0, 1, 3]].double()
    torch.testing.assert_close(d[1][keep].double(), p * (gg - (gg * p).sum()), rtol=0, atol=1e-5)


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False),
                                          ("sigmoid", True), ("sigmoid", False)])
def test_gradient_against_differences(score, renorm):
    # scores a tenth apart in a random order: a step of 1e-2 changes no choice.
    # Central differences: h^2/6 |f'''| <= 2e-5 |g|, rounding of the weights
    # 2 * 1.2e-7 / 2e-2 = 1.2e-5 each, 4 of them: within 2e-4.
    e, k, h = 12, 4, 1e-2
    g = torch.Generator().manual_seed(8)
    z = (0.1 * torch.randperm(e, generator=g).float() - 0.5)[None].cuda()
    gw = (torch.rand((1, k), generator=g) * 2 - 1).cuda()
    cfg, idx, w = run(z, k, score, renorm)
    d = torch.empty_like(z)
    ep.ep_route_backward(cfg, z, idx, gw, d)
    for j in range(e):
        zz = z.repeat(2, 1)
        zz[0, j] += h
        zz[1, j] -= h
        _, i2, w2 = run(zz, k, score, renorm)
        assert torch.equal(i2[0], idx[0]) and torch.equal(i2[1], idx[0])
        step = (zz[0, j] - zz[1, j]).double()
        num = ((w2[0] - w2[1]).double() * gw[0].double()).sum() / step
        assert abs(num - d[0, j].double()) < 2e-4, (j, num, d[0, j])


def test_long_batch_and_other_stream():
    z = logits(70001, 33)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cfg = ep.make_route_cfg(33, 5)
    idx = torch.empty((70001, 5), dtype=torch.int64, device="cuda")
    w = torch.empty((70001, 5), device="cuda")
    torch.cuda.synchronize()
    ep.ep_route(cfg, z, idx, w, stream=s)
    s.synchronize()
    top, at = torch.sort(z, dim=1, descending=True, stable=True)
    assert torch.equal(idx, at[:, :5])
    torch.testing.assert_close(w.double(), torch.softmax(top[:, :5].double(), 1), rtol=1e-5, atol=0)
    assert torch.equal(run(z, 5, "softmax", True)[2], w)


def test_the_outputs_feed_layout_and_combine():
    n, e, k, h = 128, 32, 4, 1024
    z = logits(n, e)
    cfg, idx, w = run(z, k, "softmax", True)
    hd = ep.EpHandle(ep.make_cfg(4, h, 32, 8, k))
    hd.layout(idx)
    x = torch.randn((n, h), device="cuda").bfloat16()
    recv = torch.zeros((ep.ep_recv_capacity(hd.cfg), h), dtype=torch.bfloat16, device="cuda")
    hd.dispatch(x, recv)
    out = torch.empty_like(x)
    hd.combine(recv, w, out)       # identity experts and weights that sum to 1
    assert hd.status() == 0
    torch.testing.assert_close(out.float(), x.float(), rtol=2.0 ** -7, atol=1e-6)
    hd.free()
