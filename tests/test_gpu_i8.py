"""The int8 path against plain implementations: rows to int8 bit for bit (fp32 division and
rounding as IEEE has them), products against 64 bits.

Products: whole numbers below 2^24 are exact, then two fp32 multiplications: 2 2^-24 of the
value, and 2^-8 of it where it is rounded to bf16.  Larger sums may lose 2^-23 of
the largest partial sum at each of cols/16 additions.  Gated: with g and u off by e = 2^-23 (relative)
act(g) is off by 1.13 |g| e (the slope of silu and gelu is below 1.13) and by its own
arithmetic, under 16 units of 2^-24 of |g| (the tanh form cancels against 1, so not of act(g))."""
import math

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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ---------------------------------------------------------------- rows

def rows_reference(x):
    v = x.float().cpu().numpy()
    with np.errstate(all="ignore"):
        amax = np.abs(v).max(1)
        fine = np.isfinite(v).all(1)
        s = np.where(fine, amax / np.float32(127), np.float32(np.nan)).astype(np.float32)
        q = np.where(s[:, None] > 0, v / s[:, None], 0)
        q = np.where(fine[:, None], np.clip(np.rint(q), -127, 127), 0).astype(np.int8)
    return torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()


def check_rows(x):
    q = torch.full(x.shape, 55, dtype=torch.int8, device="cuda")
    s = torch.full((x.shape[0],), -1.0, device="cuda")
    ep.ep_i8_quantize(x, q, s)
    want_q, want_s = rows_reference(x)
    assert torch.equal(s.view(torch.int32)[~torch.isnan(want_s)], want_s.view(torch.int32)[~torch.isnan(want_s)])
    assert torch.equal(torch.isnan(s), torch.isnan(want_s))
    assert torch.equal(q, want_q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,cols", [(1, 16), (5, 32), (33, 1008), (7, 1024), (9, 1040), (130, 2048), (3, 2064), (11, 4112),
                                    (64, 7168), (5, 8208), (17, 14336), (4, 16384), (3, 16400), (2, 65536)])
def test_rows(n, cols, dtype):
    x = torch.randn((n, cols), device="cuda", generator=gen(n + cols)) * torch.exp(
        3 * torch.randn((n, 1), device="cuda", generator=gen(cols)))
    check_rows(x.to(dtype))


def test_rows_on_ties_and_at_the_ends():
    """Quotients on and next to every tie, subnormal and huge rows, zeros, infinities, NaN."""
    ties = torch.arange(-127, 127, device="cuda").float() + 0.5
    row = torch.cat([torch.tensor([127.0, -127.0], device="cuda"), ties])
    x = torch.zeros((40, 272), device="cuda")
    for i, f in enumerate([1.0, 2.0 ** -20, 3.0, 0.1, 1.7e-5, 2.0 ** 100, 1e-38, 2.0 ** -140, 1.3]):
        x[3 * i, :256] = row * f
        x[3 * i + 1, :256] = torch.nextafter(row * f, torch.full_like(row, math.inf))
        x[3 * i + 2, :256] = torch.nextafter(row * f, torch.full_like(row, -math.inf))
    x[28, 5] = 2.0 ** -149
    x[29, 7] = -190 * 2.0 ** -149
    x[30] = torch.finfo(torch.float32).max
    x[31, 3] = math.inf
    x[32, 4] = -math.inf
    x[33, 271] = math.nan
    x[34, :2] = torch.tensor([math.inf, math.nan], device="cuda")
    check_rows(x)
    check_rows(x.bfloat16())
    check_rows(x[:0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_row_strides_and_alignment(dtype):
    wide = torch.randn((50, 330), device="cuda", generator=gen(1)).to(dtype)
    for a in (0, 1, 2, 4, 7, 8):
        check_rows(wide[:, a:a + 320])
    check_rows(wide[7:8, 1:17])
    check_rows(wide[::3, :64])


# ------------------------------------------------------- handles and dispatch

def handle(n, experts, topk, align, hidden=64, world=1, masked=0.1, seed=0, no_expand=False, per=None):
    g = gen(seed + n)
    z = torch.randn((n, experts), device="cuda", generator=g)
    idx = torch.topk(z, topk, dim=1).indices if n else torch.empty((0, topk), dtype=torch.int64, device="cuda")
    idx = idx.masked_fill(torch.rand((n, topk), device="cuda", generator=g) < masked, -1).contiguous()
    h = ep.EpHandle(ep.make_cfg(world, hidden, per or max(1, -(-n // world)), experts // world, topk, align, "bf16",
                                not no_expand, no_expand))
    h.layout(idx)
    return h, idx


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,experts,topk,align,hidden,no_expand", [
    (1, 4, 2, 1, 64, False), (100, 16, 4, 8, 1040, False), (77, 32, 16, 16, 2048, False), (300, 8, 1, 128, 7168, False),
    (50, 16, 8, 1, 256, True), (0, 8, 2, 8, 64, False)])
def test_dispatch(n, experts, topk, align, hidden, no_expand, dtype):
    h, _ = handle(n, experts, topk, align, hidden, world=4, no_expand=no_expand)
    x = torch.randn((n, hidden), device="cuda", generator=gen(3)).to(dtype)
    R = h.recv_capacity
    q, s = torch.full((R, hidden), 77, dtype=torch.int8, device="cuda"), torch.full((R,), -9.0, device="cuda")
    ep.ep_i8_dispatch(h, x, q, s)
    want_q, want_s = torch.full_like(q, 77), torch.full_like(s, -9.0)
    if n:
        xq, xs = rows_reference(x)
        slots = h.field(ep.FIELD_SEND_SLOT).long()
        for k in range(topk):
            ok = slots[:, k] >= 0
            want_q[slots[ok, k]] = xq[ok]
            want_s[slots[ok, k]] = xs[ok]
    assert torch.equal(q, want_q) and torch.equal(s, want_s)


def test_quantize_of_receive_rows():
    h, _ = handle(90, 16, 4, 32, world=2, per=200)       # a capacity far above the rows in use
    R = h.recv_capacity
    x = torch.randn((R, 176), device="cuda", generator=gen(4))
    used = h.field(ep.FIELD_RECV_SRC_METADATA)[:, 0] >= 0
    x[~used] = math.nan
    q, s = torch.full((R, 176), 77, dtype=torch.int8, device="cuda"), torch.full((R,), -9.0, device="cuda")
    ep.ep_i8_quantize(x, q, s, only_of=h)
    want_q, want_s = rows_reference(x)
    assert torch.equal(q[used], want_q[used]) and torch.equal(s[used], want_s[used])
    assert (q[~used] == 77).all() and (s[~used] == -9).all()


# ---------------------------------------------------------------- products

def whole(shape, seed, most=127):
    return torch.randint(-most, most + 1, shape, device="cuda", generator=gen(seed)).to(torch.int8)


def scales(shape, seed):
    return torch.rand(shape, device="cuda", generator=gen(seed)) * 0.02 + 0.001


def act64(name, v):
    if name == "silu":
        return v * torch.sigmoid(v)
    return torch.nn.functional.gelu(v, approximate="tanh")


def reference(x, xs, w, ws, act):
    """The product and how far off it may be before the rounding to the output's type."""
    sums = x.double() @ w.double().T
    y = sums * ws.double() * xs.double()[:, None]
    lost = 0.0
    if sums.numel() and float((x.double().abs() @ w.double().abs().T).max()) >= 2 ** 24:
        lost = (x.shape[1] / 16) * 2.0 ** -23 * (x.double().abs() @ w.double().abs().T) * ws.double().abs() * xs.double().abs()[:, None]
    off = 2.0 ** -23 * y.abs() + lost
    if act is None:
        return y, off
    half = y.shape[1] // 2
    g, u, eg, eu = y[:, :half], y[:, half:], off[:, :half], off[:, half:]
    a = act64(act, g)
    ea = 1.13 * eg + 16 * 2.0 ** -24 * g.abs()
    return a * u, ea * u.abs() + a.abs() * eu + ea * eu + 2.0 ** -24 * (a * u).abs()


def agree(out, x, xs, w, ws, act):
    y, off = reference(x, xs, w, ws, act)
    if out.dtype == torch.bfloat16:
        off = off + 2.0 ** -8 * (y.abs() + off)
    assert ((out.double() - y).abs() <= off + 1e-37).all(), ((out.double() - y).abs() / (off + 1e-37)).max()


def check_linear(n, rows, cols, act=None, dtype=torch.bfloat16, most=127, make=whole):
    x, w = make((n, cols), n + cols, most), make((rows, cols), rows + cols, most)
    xs, ws = scales((n,), 1), scales((rows,), 2)
    out = torch.full((n, rows // 2 if act else rows), math.nan, dtype=dtype, device="cuda")
    ep.ep_i8_linear(x, xs, w, ws, out, activation=act)
    agree(out, x, xs, w, ws, act)
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,rows,cols", [
    (1, 1, 16), (1, 64, 64), (2, 17, 48), (3, 129, 80), (1, 4096, 1024), (5, 257, 2064), (8, 1000, 512), (9, 255, 144),
    (16, 640, 4096), (17, 300, 1040), (31, 70, 256), (33, 513, 336), (63, 2048, 1024), (64, 128, 7168), (65, 260, 400),
    (100, 1024, 640), (127, 511, 1264), (129, 256, 128), (200, 2000, 912), (255, 130, 256), (256, 256, 2048),
    (257, 1281, 336), (500, 384, 1600), (1023, 520, 208), (0, 64, 64), (100, 1, 16), (24, 4099, 112), (25, 90, 16),
    (40, 30001, 64), (3001, 17, 4096)])
def test_linear(n, rows, cols, dtype):
    check_linear(n, rows, cols, None, dtype)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,rows,cols", [(1, 2, 16), (1, 4096, 512), (4, 34, 96), (13, 514, 1024), (40, 258, 2048), (65, 1026, 400),
                                         (130, 256, 640), (300, 700, 1264), (513, 126, 256)])
def test_linear_gated(n, rows, cols, act, dtype):
    check_linear(n, rows, cols, act, dtype)


@pytest.mark.parametrize("n", [1, 24, 70, 260])
@pytest.mark.parametrize("cols", [1024, 65536])
def test_linear_at_the_ends_of_int8(n, cols):
    """All 127 and -128: the largest sums there are."""
    for a, b in ((127, 127), (-128, -128), (127, -128)):
        x = torch.full((n, cols), a, dtype=torch.int8, device="cuda")
        w = torch.full((40, cols), b, dtype=torch.int8, device="cuda")
        xs, ws = torch.full((n,), 2.0 ** -10, device="cuda"), torch.full((40,), 2.0 ** -10, device="cuda")
        out = torch.empty((n, 40), device="cuda")
        ep.ep_i8_linear(x, xs, w, ws, out)
        agree(out, x, xs, w, ws, None)


def test_linear_scales_that_are_not_numbers():
    x, w = whole((70, 64), 1), whole((50, 64), 2)
    xs, ws = scales((70,), 3), scales((50,), 4)
    xs[3], xs[5], ws[7], ws[8] = math.nan, 0.0, math.inf, 0.0
    for n in (10, 70):
        out = torch.empty((n, 50), device="cuda")
        ep.ep_i8_linear(x[:n], xs[:n], w, ws, out)
        want = (x[:n].double() @ w.double().T).float() * ws * xs[:n, None]
        assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(torch.isinf(out), torch.isinf(want))
        assert (out[5, torch.isfinite(want[5])] == 0).all()


def test_linear_behind_two_gigabytes():
    """Weights whose offsets pass 32 bits."""
    rows, cols = 70001, 32768
    w = torch.zeros((rows, cols), dtype=torch.int8, device="cuda")
    at = torch.tensor([0, 1, 65535, 65536, 65537, 69000, 70000], device="cuda")
    w[at] = whole((7, cols), 5, 9)
    ws = scales((rows,), 2)
    for n in (2, 150):
        x, xs = whole((n, cols), 6, 9), scales((n,), 1)
        out = torch.empty((n, rows), dtype=torch.bfloat16, device="cuda")
        ep.ep_i8_linear(x, xs, w, ws, out)
        agree(out[:, at], x, xs, w[at], ws[at], None)
        out[:, at] = 0
        assert (out == 0).all()


def check_grouped(h, rows, cols, act, dtype, seed=0):
    E, R = h.cfg.world_size * h.cfg.num_expert_per_rank, h.recv_capacity
    x, w = whole((R, cols), seed + 1), whole((E, rows, cols), seed + 2)
    xs, ws = scales((R,), seed + 3), scales((E, rows), seed + 4)
    used = h.field(ep.FIELD_RECV_SRC_METADATA)[:, 0] >= 0
    xs[~used] = math.nan                                  # what padding rows hold does not matter
    out = torch.full((R, rows // 2 if act else rows), 7.0, dtype=dtype, device="cuda")
    ep.ep_i8_grouped(h, x, xs, w, ws, out, activation=act)
    assert (out[~used] == 7).all()
    first, count = h.field(ep.FIELD_PSUM_PER_EXPERT).tolist(), h.field(ep.FIELD_NUM_UNALIGNED_PER_EXPERT).tolist()
    for e in range(E):
        a, b = first[e], first[e] + count[e]
        if count[e]:
            agree(out[a:b], x[a:b], xs[a:b], w[e], ws[e], act)


@pytest.mark.parametrize("act", [None, "silu", "gelu_tanh"])
@pytest.mark.parametrize("n,experts,topk,align,rows,cols,dtype", [
    (1, 4, 2, 1, 64, 64, torch.bfloat16), (7, 16, 3, 8, 130, 272, torch.float32), (64, 8, 2, 16, 1000, 512, torch.bfloat16),
    (300, 6, 6, 1, 258, 144, torch.bfloat16), (900, 12, 4, 128, 514, 640, torch.float32), (33, 64, 1, 4, 32, 1040, torch.bfloat16),
    (1500, 4, 4, 64, 256, 256, torch.bfloat16), (2, 2048, 16, 1, 16, 16, torch.bfloat16), (0, 8, 2, 8, 64, 64, torch.bfloat16)])
def test_grouped(n, experts, topk, align, rows, cols, dtype, act):
    h, _ = handle(n, experts, topk, align)
    check_grouped(h, rows, cols, act, dtype)


@pytest.mark.parametrize("shares", [[0, 0, 0, 1000], [1000, 0, 1, 0], [1, 257, 0, 300], [16, 16, 16, 16], [255, 256, 257, 512],
                                    [0, 0, 0, 0]])
def test_grouped_routings(shares):
    """Experts without rows, with one, with whole and ragged tiles."""
    ids = torch.repeat_interleave(torch.arange(4), torch.tensor(shares)).cuda()[:, None]
    n = max(1, ids.shape[0])
    h = ep.EpHandle(ep.make_cfg(1, 64, 2 * n, 4, 1, 8, "bf16", True))
    if ids.shape[0] == 0:
        ids = torch.full((1, 1), -1, dtype=torch.int64, device="cuda")
    h.layout(ids.contiguous())
    for act in (None, "silu"):
        check_grouped(h, 320, 400, act, torch.bfloat16)


def test_grouped_behind_two_gigabytes():
    """Experts whose weights begin past 32 bits of bytes."""
    E, rows, cols = 40, 4096, 16384
    w = torch.zeros((E, rows, cols), dtype=torch.int8, device="cuda")
    for e in (0, 31, 32, 39):
        w[e] = whole((rows, cols), e, 9)
    ws = scales((E, rows), 1)
    h, _ = handle(90, E, 2, 8, masked=0.0)
    x, xs = whole((h.recv_capacity, cols), 2, 9), scales((h.recv_capacity,), 3)
    out = torch.zeros((h.recv_capacity, rows), dtype=torch.bfloat16, device="cuda")
    ep.ep_i8_grouped(h, x, xs, w, ws, out)
    first, count = h.field(ep.FIELD_PSUM_PER_EXPERT).tolist(), h.field(ep.FIELD_NUM_UNALIGNED_PER_EXPERT).tolist()
    for e in range(E):
        a, b = first[e], first[e] + count[e]
        if e in (0, 31, 32, 39):
            agree(out[a:b], x[a:b], xs[a:b], w[e], ws[e], None)
        else:
            assert (out[a:b] == 0).all()


def test_products_in_a_graph_on_two_streams():
    """Captured products replayed beside eager ones on another stream: equal bits."""
    calls = []
    for n in (1, 40, 300):
        x, w, xs, ws = whole((n, 1024), n), whole((512, 1024), 9), scales((n,), 1), scales((512,), 2)
        calls.append((x, xs, w, ws))
    h, _ = handle(200, 8, 2, 16)
    gx, gw = whole((h.recv_capacity, 256), 1), whole((8, 192, 256), 2)
    gxs, gws = scales((h.recv_capacity,), 3), scales((8, 192), 4)

    def run():
        outs = []
        for x, xs, w, ws in calls:
            out = torch.zeros((x.shape[0], 512), dtype=torch.bfloat16, device="cuda")
            ep.ep_i8_linear(x, xs, w, ws, out)
            outs.append(out)
        out = torch.zeros((h.recv_capacity, 192), dtype=torch.bfloat16, device="cuda")
        ep.ep_i8_grouped(h, gx, gxs, gw, gws, out)
        return outs + [out]
    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        captured = run()
    torch.cuda.synchronize()
    for _ in range(10):
        graph.replay()
        with torch.cuda.stream(side):
            eager = run()
    torch.cuda.synchronize()
    for got in (captured, eager):
        assert all(torch.equal(a, b) for a, b in zip(got, first))
    assert ep.ep_i8_status() == 0


def test_experts_end_to_end():
    """Layout, int8 dispatch, gate and up products, int8 rows, down products, combine, each against the plain
    form of its own inputs; the whole against unquantised experts: a row's rounding is at most half a step of
    amax/127, uniform in it (rms 0.29 of a step), and a normal row's amax is at most 6 deviations, so each
    quantised factor is off by 1.4% rms; five of them (x, w13 twice, h, w2) and two bf16 roundings are
    off by 4% of the output together."""
    n, H, I, E, K = 300, 512, 256, 16, 4
    g = gen(11)
    h, idx = handle(n, E, K, 16, hidden=H, masked=0.0)
    x = torch.randn((n, H), device="cuda", generator=g).bfloat16()
    w13 = torch.randn((E, 2 * I, H), device="cuda", generator=g) * H ** -0.5
    w2 = torch.randn((E, H, I), device="cuda", generator=g) * I ** -0.5
    tw = torch.rand((n, K), device="cuda", generator=g)

    def quantised(w):
        q, s = torch.empty(w.shape, dtype=torch.int8, device="cuda"), torch.empty(w.shape[:2], device="cuda")
        ep.ep_i8_quantize(w.flatten(0, 1), q.view(-1, w.shape[2]), s.view(-1))
        return q, s
    q13, s13 = quantised(w13)
    q2, s2 = quantised(w2)
    R = h.recv_capacity
    xq, xs = torch.empty((R, H), dtype=torch.int8, device="cuda"), torch.empty((R,), device="cuda")
    hid = torch.empty((R, I), dtype=torch.bfloat16, device="cuda")
    hq, hs = torch.empty((R, I), dtype=torch.int8, device="cuda"), torch.empty((R,), device="cuda")
    y, out = torch.empty((R, H), dtype=torch.bfloat16, device="cuda"), torch.empty((n, H), device="cuda")
    ep.ep_i8_dispatch(h, x, xq, xs)
    ep.ep_i8_grouped(h, xq, xs, q13, s13, hid, activation="silu")
    ep.ep_i8_quantize(hid, hq, hs, only_of=h)
    ep.ep_i8_grouped(h, hq, hs, q2, s2, y)
    h.combine(y, tw, out)
    first, count = h.field(ep.FIELD_PSUM_PER_EXPERT).tolist(), h.field(ep.FIELD_NUM_UNALIGNED_PER_EXPERT).tolist()
    for e in range(E):
        a, b = first[e], first[e] + count[e]
        agree(hid[a:b], xq[a:b], xs[a:b], q13[e], s13[e], "silu")
        agree(y[a:b], hq[a:b], hs[a:b], q2[e], s2[e], None)
    want = torch.zeros((n, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, k = (idx == e).nonzero(as_tuple=True)
        u = x[t].double() @ w13[e].double().T
        v = (torch.nn.functional.silu(u[:, :I]) * u[:, I:]) @ w2[e].double().T
        want.index_add_(0, t, v * tw[t, k, None].double())
    assert ((out - want).norm() / want.norm()).item() < 0.04
    assert h.status() == 0 and ep.ep_i8_status() == 0
