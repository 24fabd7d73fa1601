"""The router's training losses against a plain implementation in 64 bits.

Tolerances, in units of 2^-24 (half a step of fp32).  A probability is exp of a
difference (its rounding moves the exponent by |z - peak| < 64 units, expf by 4),
over a sum (E/32 + 5 additions at most 7 + 64 units here) with two more
roundings: under 256 units of its value, 2^-16.  The sums over tokens only add positive
values: a warp's chain, 8 warps, a block's rows, together under 256 additions more:
2^-15 of the value, elementwise, and the same for the losses.  The gradient is a
difference c - sum c p of terms of at most max|c - mean|: 2^-15 of
share p max|c - mean| + rise p, and half a step of the output's type.  Tiny values are
let go below 1e-30."""
import math

import pytest
import torch

import combine_ep_layout_gb300 as ep

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -15


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def make(n, experts, topk, dtype=torch.float32, masked=0.0, seed=0, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * n + experts)
    z = spread * torch.randn((n, experts), device="cuda", generator=g) + torch.randn((1, experts), device="cuda", generator=g)
    z = z.masked_fill(torch.rand((n, experts), device="cuda", generator=g) < masked, -math.inf).to(dtype)
    idx = torch.full((n, topk), -1, dtype=torch.int64, device="cuda")
    if n:
        ep.ep_route(ep.make_route_cfg(experts, topk), z, idx, torch.empty((n, topk), device="cuda"))
    return z, idx


def reference(z, idx, offsets, experts, topk, sigmoid):
    """counts, sums, tokens, the losses and, as functions of the scores' gradient, p and lse, in 64 bits."""
    n, m = z.shape[0], len(offsets) - 1
    z = torch.where(torch.isnan(z), -math.inf, z.double())
    valid = (idx >= 0) & (idx < experts)
    live = valid.any(1)
    masked = ~(z > -math.inf)
    empty = masked.all(1)
    soft = torch.where(masked | empty[:, None], 0.0, torch.softmax(torch.where(empty[:, None], 0.0, z), 1))
    if sigmoid:
        peak = z.amax(1, keepdim=True).clamp_max(0)
        peak = torch.where(peak > -math.inf, peak, 0.0)
        s = torch.where(masked, 0.0, torch.exp(z - peak) / (1 + torch.exp(z)))
        s = torch.where(z >= 0, torch.sigmoid(z), s)     # peak is 0 there
        p = s / s.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        p = soft
    lse = torch.where(empty, 0.0, torch.logsumexp(torch.where(empty[:, None], 0.0, z), 1))
    counts = torch.zeros((m, experts), dtype=torch.int32, device=z.device)
    sums = torch.zeros((m, experts), dtype=torch.float64, device=z.device)
    tokens = torch.zeros((m + 1,), dtype=torch.int32, device=z.device)
    of = torch.full((n,), -1, device=z.device)
    for g in range(m):
        a, b = offsets[g], offsets[g + 1]
        if b <= a:
            continue
        of[a:b] = g
        ids = idx[a:b][valid[a:b]]
        counts[g] = torch.bincount(ids, minlength=experts).int()
        sums[g] = (p[a:b] * live[a:b, None]).sum(0)
        tokens[g] = int(live[a:b].sum())
    tokens[m] = tokens[:m].sum()
    live &= of >= 0
    t = tokens[:m].double().clamp_min(1)
    share = experts / (topk * m * t * t)
    loss = torch.stack([((counts * sums).sum(1) * share).sum(),
                        (lse.square() * live).sum() / max(1, int(tokens[m]))])
    return dict(counts=counts, sums=sums, tokens=tokens, loss=loss, p=p, soft=soft, lse=lse, live=live, of=of,
                share=share, z=z, masked=masked)


def gradient(r, grad_loss, sigmoid):
    of = r["of"].clamp_min(0)
    c = r["counts"].double()[of]
    gb, gz = [float(v) for v in grad_loss]
    p = r["p"]
    share = gb * r["share"][of][:, None]
    d = share * p * (c - (c * p).sum(1, keepdim=True))
    if sigmoid:
        d = d * torch.sigmoid(-r["z"])
    rise = gz * 2.0 / max(1, int(r["tokens"][-1])) * r["lse"][:, None]
    d = d + rise * r["soft"]
    mean = (c * p).sum(1, keepdim=True)
    size = abs(gb) * r["share"][of][:, None] * p * (c - mean).abs().amax(1, keepdim=True) + rise.abs() * r["soft"]
    keep = r["live"][:, None] & ~r["masked"]
    return torch.where(keep, d, 0.0), torch.where(keep, size, 0.0)


def outputs(m, experts):
    return (torch.full((m, experts), -5, dtype=torch.int32, device="cuda"), torch.full((m, experts), math.nan, device="cuda"),
            torch.full((m + 1,), -5, dtype=torch.int32, device="cuda"), torch.full((2,), math.nan, device="cuda"))


def check(z, idx, offsets, topk, score, grad=True, balance=None):
    n, experts = z.shape
    m = len(offsets) - 1
    given = None if offsets == [0, n] else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    b = balance or ep.EpBalance(ep.make_route_cfg(experts, topk, score), max(1, n), m)
    counts, sums, tokens, loss = outputs(m, experts)
    b.forward(z, idx, counts, sums, tokens, loss, seq_offsets=given)
    r = reference(z, idx, offsets, experts, topk, score == "sigmoid")
    assert torch.equal(counts, r["counts"]) and torch.equal(tokens, r["tokens"])
    assert ((sums - r["sums"]).abs() <= TOL * r["sums"] + 1e-30).all()
    over = r["loss"] > torch.finfo(torch.float32).max      # a row at the type's lowest value: its lse^2 is 1e76
    assert torch.isinf(loss[over]).all()
    assert ((loss - r["loss"]).abs() <= TOL * r["loss"] + 1e-30)[~over].all(), (loss, r["loss"])
    if not grad:
        return
    gl = torch.tensor([0.7, -0.3], device="cuda")
    want, size = gradient(r, gl, score == "sigmoid")
    out = torch.full_like(z, 3.0)
    b.backward(z, idx, counts, tokens, gl, out, seq_offsets=given)
    inside = (r["of"] >= 0)[:, None]
    want = torch.where(inside, want, 3.0)
    half = torch.finfo(z.dtype).eps / 2
    bound = TOL * size + half * want.abs() + 1e-30
    off = (out.double() - want).abs()
    assert (off <= bound).all(), (off / bound).max()
    # added to what is there, in fp32
    base = torch.randn_like(z.float()).to(z.dtype)
    more = base.clone()
    b.backward(z, idx, counts, tokens, gl, more, seq_offsets=given, accumulate=True)
    want = torch.where(inside, base.double() + torch.where(inside, want, 0.0), base.double())
    assert ((more.double() - want).abs() <= TOL * size + (half + 2.0 ** -24) * want.abs() + 2.0 ** -24 * base.double().abs() + 1e-30).all()


SIZES = [(1, 1, 1), (1, 8, 8), (3, 33, 4), (64, 64, 8), (257, 250, 7), (1000, 129, 6), (4099, 256, 8), (300, 511, 16),
         (130, 1024, 8), (67, 2048, 16), (9, 1361, 3)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,experts,topk", SIZES)
def test_one_sequence(n, experts, topk, dtype, score):
    z, idx = make(n, experts, topk, dtype)
    check(z, idx, [0, n], topk, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("offsets", [[0, 700], [0, 0, 1, 1, 1, 350, 699, 700], [5, 5, 5], [13, 64, 64, 65, 690],
                                     [0] + [1] * 40 + [700], list(range(0, 701, 10)), list(range(0, 701))])
def test_sequences(offsets, score):
    z, idx = make(700, 60, 4, masked=0.2)
    idx[::7] = -1                                        # padding
    check(z, idx, offsets, 4, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_rows_and_strange_ids(score):
    z, idx = make(90, 40, 6, masked=0.9)
    z[10] = -math.inf                                    # nothing left: ep_route gives -1 only
    idx[10] = -1
    z[11] = -math.inf                                    # nothing left although ids are there
    z[12, 3] = math.nan
    z[13] = -300.0                                       # sigmoids that all underflow
    z[14] = 80.0
    z[15] = torch.finfo(torch.float32).min               # a mask by the lowest value
    idx[20] = torch.tensor([-1, 40, 3, 3, 1 << 40, -(1 << 40)], device="cuda")     # twice the same, outside
    check(z, idx, [0, 90], 6, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_no_live_token(score):
    z, idx = make(40, 16, 2)
    idx.fill_(-1)
    check(z, idx, [0, 40], 2, score)
    check(z[:0], idx[:0], [0, 0], 2, score, grad=False)


def test_infinite_scores():
    z, idx = make(4, 8, 2)
    z[0, 3] = math.inf
    z[1, 2] = z[1, 6] = math.inf
    b = ep.EpBalance(ep.make_route_cfg(8, 2), 4)
    counts, sums, tokens, loss = outputs(1, 8)
    b.forward(z[:2], idx[:2], counts, sums, tokens, loss)
    assert sums[0].tolist() == [0, 0, 0.5, 1.0, 0, 0, 0.5, 0] and math.isinf(loss[1].item())
    assert math.isfinite(loss[0].item())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_alignment(dtype):
    wide, idx = make(200, 67, 4, dtype)
    for a, w in ((0, 64), (1, 64), (3, 61), (0, 67)):
        z = wide[:, a:a + w]
        ids = torch.where(idx < w, idx, -1)
        check(z, ids, [0, 200], 4, "softmax")
    one = wide[5:6, :64].expand(1, 64)
    check(one, torch.where(idx[5:6] < 64, idx[5:6], -1), [0, 1], 4, "sigmoid")
    # a gradient with a row stride of its own
    z = wide[:, :64]
    ids = torch.where(idx < 64, idx, -1)
    b = ep.EpBalance(ep.make_route_cfg(64, 4), 200)
    counts, sums, tokens, loss = outputs(1, 64)
    b.forward(z, ids, counts, sums, tokens, loss)
    gl = torch.tensor([1.0, 1.0], device="cuda")
    flat, strided = torch.empty((200, 64), dtype=dtype, device="cuda"), torch.full((200, 70), 9.0, dtype=dtype, device="cuda")
    b.backward(z, ids, counts, tokens, gl, flat)
    b.backward(z, ids, counts, tokens, gl, strided[:, 3:67])
    assert torch.equal(strided[:, 3:67], flat) and (strided[:, :3] == 9).all() and (strided[:, 67:] == 9).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(score):
    """The losses with the counts held fixed, moved along a direction by +-h: central differences of
    the 64-bit losses are off by h^2 (1e-8 of the losses' size) and by the kernel's 2^-15."""
    z, idx = make(50, 24, 3, spread=2.0)
    offsets = [0, 20, 50]
    b = ep.EpBalance(ep.make_route_cfg(24, 3, score), 50, 2)
    counts, sums, tokens, loss = outputs(2, 24)
    given = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    b.forward(z, idx, counts, sums, tokens, loss, seq_offsets=given)
    way = torch.randn((50, 24), dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    for gl in ([1.0, 0.0], [0.0, 1.0]):
        out = torch.empty_like(z)
        b.backward(z, idx, counts, tokens, torch.tensor(gl, device="cuda"), out, seq_offsets=given)
        h = 1e-4
        up = reference(z.double() + h * way, idx, offsets, 24, 3, score == "sigmoid")["loss"]
        down = reference(z.double() - h * way, idx, offsets, 24, 3, score == "sigmoid")["loss"]
        slope = float(((up - down) / (2 * h) * torch.tensor(gl, device="cuda")).sum())
        terms = out.double() * way
        assert abs(float(terms.sum()) - slope) <= TOL * float(terms.abs().sum()) + 1e-6 * float(loss.sum())


def test_equal_bits_and_replays():
    """Forward and backward captured on a stream of their own and replayed on new scores give the bits of
    plain calls; so does a second handle at the same time."""
    n, experts, topk = 5000, 128, 8
    z, idx = make(n, experts, topk)
    z2, idx2 = make(n, experts, topk, seed=1)
    cfg = ep.make_route_cfg(experts, topk)
    gl = torch.tensor([1.0, 0.1], device="cuda")

    def run(b, z, idx, o, grad):
        b.forward(z, idx, *o)
        b.backward(z, idx, o[0], o[2], gl, grad)
    first, grad = outputs(1, experts), torch.empty_like(z)
    b = ep.EpBalance(cfg, n)
    run(b, z, idx, first, grad)
    zc, ic, o, gc = z2.clone(), idx2.clone(), outputs(1, experts), torch.empty_like(z)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        run(b, zc, ic, o, gc)
    zc.copy_(z), ic.copy_(idx)
    other, out2, grad2 = ep.EpBalance(cfg, n), outputs(1, experts), torch.empty_like(z)
    torch.cuda.synchronize()
    for _ in range(20):
        graph.replay()
        with torch.cuda.stream(side):
            run(other, z, idx, out2, grad2)
    torch.cuda.synchronize()
    for got in (o, out2):
        assert all(torch.equal(x, y) for x, y in zip(got, first))
    assert torch.equal(gc, grad) and torch.equal(grad2, grad)


def test_a_smaller_batch_than_the_handle_and_many_tokens():
    n, experts, topk = 70000, 48, 4
    z, idx = make(n, experts, topk)
    b = ep.EpBalance(ep.make_route_cfg(experts, topk), n, 9)
    check(z[:33], idx[:33], [0, 33], topk, "softmax", balance=b)
    check(z, idx, [0, n], topk, "softmax", balance=b)
    check(z, idx, [7, 9000, 9000, 69999], topk, "softmax", balance=b)
