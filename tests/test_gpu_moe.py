"""The MoE layer for a few tokens against a plain implementation in 64 bits.

Exact inputs: gates of 64 (silu(64) is 64 in fp32), whole-number up projections
and down weights, weights that are powers of two: the result is exact in fp32.
Random inputs: h is rounded to bf16 once, an error of at most 2^-8 of each h,
independent of one another: with sigma = 2^-8 / sqrt(3) the 2-norm over (k, i) of
w_k W2 h times 8 sigma, plus 2^-19 of the sum of absolute products for the fp32
sums of both products, plus 2^-8 of the value for a bf16 output.
"""
import pytest
import torch

import combine_ep_layout_gb300 as ep

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def dense(q, s):
    if s is None:
        return q.double()
    w = torch.empty((*q.shape[:-1], 2 * q.shape[-1]), dtype=torch.float64, device=q.device)
    w[..., 0::2] = (q & 15).double() - 8
    w[..., 1::2] = (q >> 4).double() - 8
    return w * s.double().repeat_interleave(w.shape[-1] // s.shape[-1], -1)


def act64(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh((2.0 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)))


def reference(x, idx, w, wt, act="silu", bias=None):
    """(out, tolerance without the output's rounding) in 64 bits."""
    w13, w2, s13, s2 = wt.tensors
    E, I = w13.shape[0], w13.shape[1] // 2
    y = torch.zeros((x.shape[0], w2.shape[1]), dtype=torch.float64, device="cuda")
    var, mag = torch.zeros_like(y), torch.zeros_like(y)
    for e in range(E):
        t, k = (idx == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        a = dense(w13[e], None if s13 is None else s13[e])
        b = dense(w2[e], None if s2 is None else s2[e])
        u = x[t].double() @ a.T
        h = act64(u[:, :I], act) * u[:, I:]
        m = x[t].double().abs() @ a.abs().T
        hm = 1.2 * m[:, :I] * u[:, I:].abs() + act64(u[:, :I], act).abs() * m[:, I:]
        c = w[t, k].double()[:, None]
        y.index_add_(0, t, c * (h @ b.T))
        var.index_add_(0, t, c ** 2 * (h ** 2 @ (b ** 2).T))
        mag.index_add_(0, t, c.abs() * ((h.abs() + hm) @ b.abs().T))
    if bias is not None:
        y += bias.double()
    return y, 8 * 2.0 ** -8 / 3 ** 0.5 * var.sqrt() + 2.0 ** -19 * mag


def make(E, H, I, weights="bf16", group=0, seed=0, exact=False):
    g = torch.Generator(device="cuda").manual_seed(seed + E * 7 + H * 3 + I)

    def one(rows, cols):
        if weights == "bf16":
            return (torch.randn((E, rows, cols), device="cuda", generator=g) * cols ** -0.5).bfloat16(), None
        q = torch.randint(0, 256, (E, rows, cols // 2), dtype=torch.uint8, device="cuda", generator=g)
        s = (torch.rand((E, rows, cols // group), device="cuda", generator=g) + 0.5) / (4.6 * cols ** 0.5)
        return q, s
    w13, s13 = one(2 * I, H)
    w2, s2 = one(H, I)
    if exact:
        # x[:, 0] is 1 and the gate reads it alone; the up projection reads columns 1..7
        if weights == "bf16":
            w13.zero_()
            w13[:, :I, 0] = 64.0
            w13[:, I:, 1:8] = torch.randint(-2, 3, (E, I, 7), device="cuda", generator=g).bfloat16()
            w2.copy_(torch.randint(-2, 3, w2.shape, device="cuda", generator=g))
        else:
            w13.fill_(0x88)
            w13[:, :I, 0] = 0x8c                                # nibble 12: 4 * 16
            w13[:, I:, 1:4] = torch.randint(0, 256, (E, I, 3), dtype=torch.uint8, device="cuda", generator=g)
            s13.fill_(0.25)
            s13[:, :I] = 16.0
            s2.copy_(2.0 ** torch.randint(-2, 2, s2.shape, device="cuda", generator=g).float())
    return ep.EpMoeWeights(w13, w2, s13, s2)


def tokens(n, H, E, K, seed=0, exact=False):
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * n + H)
    if exact:
        x = torch.zeros((n, H), device="cuda")
        x[:, 0] = 1.0
        x[:, 1:8] = torch.randint(-1, 2, (n, 7), device="cuda", generator=g).float()
        w = 2.0 ** torch.randint(-2, 2, (n, K), device="cuda", generator=g).float()
    else:
        x = torch.randn((n, H), device="cuda", generator=g)
        w = torch.rand((n, K), device="cuda", generator=g)
    idx = torch.rand((n, max(E, K)), device="cuda", generator=g).argsort(1)[:, :K] % E
    return x.bfloat16(), idx.contiguous(), w


def handle(E, H, I, K, weights="bf16", group=0, act="silu", max_tokens=64):
    return ep.EpMoe(ep.make_moe_cfg(H, I, E, K, max_tokens, weights, group, act))


def check(m, x, idx, w, wt, act="silu", bias=None, dtype=torch.bfloat16, exact=False):
    out = torch.full((x.shape[0], m.cfg.hidden_dim), float("nan"), dtype=dtype, device="cuda")
    m.forward(x, idx, w, wt, out, bias=bias)
    ref, tol = reference(x, idx, w, wt, act, bias)
    if exact:
        assert torch.equal(out, ref.to(dtype))
    else:
        if dtype == torch.bfloat16:
            tol = tol + 2.0 ** -7.99 * ref.abs()
        else:
            tol = tol + 2.0 ** -22 * ref.abs()
        bad = ~((out.double() - ref).abs() <= tol)
        assert not bad.any(), (bad.sum().item(), (out.double() - ref).abs().max().item())
    return out


#       n   K   E    H     I
BF16 = [(1, 1, 1, 8, 8), (1, 8, 64, 1024, 512), (2, 2, 8, 72, 24), (3, 4, 60, 520, 136), (4, 4, 32, 1024, 512),
        (7, 1, 4, 64, 264), (8, 2, 2, 264, 64), (9, 6, 128, 1000, 40), (16, 16, 16, 136, 72),
        (17, 3, 257, 256, 128), (31, 8, 64, 512, 256), (33, 2, 8, 2048, 1000), (64, 8, 64, 776, 328),
        (64, 1, 1, 128, 128), (64, 2, 3, 384, 640), (5, 2, 2048, 16, 16), (1, 16, 20, 4104, 16),
        (40, 4, 16, 16, 2056)]
INT4 = [(1, 1, 1, 32, 32, 32), (1, 8, 64, 1024, 512, 128), (2, 2, 8, 96, 64, 32), (3, 4, 60, 512, 192, 64),
        (4, 4, 32, 1024, 512, 32), (7, 1, 4, 128, 256, 128), (8, 2, 2, 320, 64, 64), (9, 6, 128, 1024, 96, 32),
        (16, 16, 16, 160, 96, 32), (17, 3, 257, 256, 128, 128), (31, 8, 64, 512, 256, 64),
        (33, 2, 8, 2048, 1024, 128), (64, 8, 64, 768, 384, 128), (64, 1, 1, 128, 128, 64),
        (64, 2, 3, 384, 640, 128), (5, 2, 2048, 32, 32, 32), (40, 4, 16, 32, 2080, 32)]


@pytest.mark.parametrize("n,K,E,H,I", BF16)
def test_bf16_weights(n, K, E, H, I):
    m, wt = handle(E, H, I, K), make(E, H, I)
    x, idx, w = tokens(n, H, E, K)
    check(m, x, idx, w, wt)
    check(m, x, idx, w, wt, dtype=torch.float32)
    assert m.status() == 0


@pytest.mark.parametrize("n,K,E,H,I", BF16)
def test_bf16_weights_exact(n, K, E, H, I):
    m, wt = handle(E, H, I, K), make(E, H, I, exact=True)
    x, idx, w = tokens(n, H, E, K, exact=True)
    check(m, x, idx, w, wt, dtype=torch.float32, exact=True)
    check(m, x, idx, w, wt, exact=True)


@pytest.mark.parametrize("n,K,E,H,I,group", INT4)
def test_4_bit_weights(n, K, E, H, I, group):
    m, wt = handle(E, H, I, K, "int4", group), make(E, H, I, "int4", group)
    x, idx, w = tokens(n, H, E, K)
    check(m, x, idx, w, wt)
    check(m, x, idx, w, wt, dtype=torch.float32)
    assert m.status() == 0


@pytest.mark.parametrize("n,K,E,H,I,group", INT4)
def test_4_bit_weights_exact(n, K, E, H, I, group):
    m, wt = handle(E, H, I, K, "int4", group), make(E, H, I, "int4", group, exact=True)
    x, idx, w = tokens(n, H, E, K, exact=True)
    check(m, x, idx, w, wt, dtype=torch.float32, exact=True)
    check(m, x, idx, w, wt, exact=True)


FORMS = [("bf16", 0), ("int4", 64)]


@pytest.mark.parametrize("weights,group", FORMS)
def test_every_number_of_tokens_on_one_handle(weights, group):
    E, H, I, K = 6, 192, 128, 3
    m, wt = handle(E, H, I, K, weights, group), make(E, H, I, weights, group, exact=True)
    x, idx, w = tokens(64, H, E, K, exact=True)
    for n in list(range(1, 65)) + [3, 64, 1]:
        check(m, x[:n].contiguous(), idx[:n].contiguous(), w[:n].contiguous(), wt, dtype=torch.float32, exact=True)


@pytest.mark.parametrize("weights,group", FORMS)
@pytest.mark.parametrize("n", [1, 10, 64])
def test_every_token_on_one_expert(n, weights, group):
    E, H, I, K = 16, 256, 192, 2
    m, wt = handle(E, H, I, K, weights, group), make(E, H, I, weights, group)
    x, idx, w = tokens(n, H, E, K)
    idx[:, 0] = 11
    check(m, x, idx, w, wt)
    idx[:] = 11                       # the same expert twice for every token
    check(m, x, idx, w, wt)
    assert m.status() == 0


@pytest.mark.parametrize("weights,group", FORMS)
def test_masked_entries(weights, group):
    E, H, I, K, n = 12, 128, 128, 4, 20
    m, wt = handle(E, H, I, K, weights, group), make(E, H, I, weights, group)
    x, idx, w = tokens(n, H, E, K)
    mask = torch.rand((n, K), device="cuda") < 0.5
    mask[3] = True                    # a token with nothing left
    mask[4] = False
    idx[mask] = -1
    clean = w.clone()
    w[mask] = float("nan")            # a masked entry's weight is not read
    bias = torch.randn((n, H), device="cuda").bfloat16()
    out = torch.empty_like(x)
    m.forward(x, idx, w, wt, out)
    assert (out[3] == 0).all()
    ref, tol = reference(x, idx, clean, wt)
    assert ((out.double() - ref).abs() <= tol + 2.0 ** -7.99 * ref.abs()).all()
    m.forward(x, idx, w, wt, out, bias=bias)
    assert torch.equal(out[3], bias[3])
    idx[:] = -1                       # nothing left at all
    m.forward(x, idx, w, wt, out)
    assert (out == 0).all()
    m.forward(x, idx, w, wt, out, bias=bias)
    assert torch.equal(out, bias)
    assert m.status() == 0


@pytest.mark.parametrize("weights,group", [("bf16", 0), ("int4", 32), ("int4", 128)])
@pytest.mark.parametrize("n", [2, 20])
def test_huge_activations(n, weights, group):
    # the columns that only the up projection reads, times 2^66: h and the output scale with them
    E, H, I, K = 6, 256, 128, 2
    m, wt = handle(E, H, I, K, weights, group), make(E, H, I, weights, group, exact=True)
    x, idx, w = tokens(n, H, E, K, exact=True)
    x[::2, 1:8] *= 2.0 ** 66
    check(m, x, idx, w, wt, dtype=torch.float32, exact=True)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("n", [2, 8, 20])
def test_tiny_up_projection(n, group):
    # its scales times 2^-80: h and the output scale with them
    E, H, I, K = 6, 256, 128, 2
    m, wt = handle(E, H, I, K, "int4", group), make(E, H, I, "int4", group, exact=True)
    wt.tensors[2][:, I:] *= 2.0 ** -80
    x, idx, w = tokens(n, H, E, K, exact=True)
    check(m, x, idx, w, wt, dtype=torch.float32, exact=True)


@pytest.mark.parametrize("weights,group", FORMS)
def test_infinite_activations_are_not_hidden(weights, group):
    E, H, I, K, n = 4, 128, 64, 1, 5
    m, wt = handle(E, H, I, K, weights, group), make(E, H, I, weights, group)
    x, idx, w = tokens(n, H, E, K)
    a, b = torch.empty_like(x), torch.empty_like(x)
    m.forward(x, idx, w, wt, a)
    bad = x.clone()
    bad[2, 5] = float("inf")
    m.forward(bad, idx, w, wt, b)
    keep = [t for t in range(n) if t != 2]
    assert torch.equal(a[keep], b[keep]) and not torch.isfinite(b[2]).any() and m.status() == 0


def test_ids_out_of_range_are_skipped_and_reported():
    E, H, I, K, n = 5, 64, 64, 3, 6
    m, wt = handle(E, H, I, K), make(E, H, I)
    x, idx, w = tokens(n, H, E, K)
    good = idx.clone()
    good[1, 2] = good[4, 0] = good[5, 1] = -1
    idx[1, 2], idx[4, 0], idx[5, 1] = 5, -2, 1 << 40
    a, b = torch.empty_like(x), torch.empty_like(x)
    m.forward(x, idx, w, wt, a)
    assert m.status() == 1 and m.status() == 0
    m.forward(x, good, w, wt, b)
    assert m.status() == 0 and torch.equal(a, b)


@pytest.mark.parametrize("weights,group", FORMS)
def test_only_active_experts_and_own_tokens_count(weights, group):
    E, H, I, K, n = 8, 128, 64, 2, 9
    m, wt = handle(E, H, I, K, weights, group), make(E, H, I, weights, group)
    x, idx, w = tokens(n, H, 6, K)                  # experts 6 and 7 are not chosen
    a, b = torch.empty_like(x), torch.empty_like(x)
    m.forward(x, idx, w, wt, a)
    for t in (wt.tensors[:2] if weights == "bf16" else wt.tensors[2:]):
        t[6:] = float("nan")
    x2 = x.clone()
    x2[4] = float("nan")
    m.forward(x2, idx, w, wt, b)
    keep = [t for t in range(n) if t != 4]
    assert torch.equal(a[keep], b[keep]) and b[4].isnan().all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_bias_and_gelu(dtype):
    E, H, I, K, n = 8, 200, 96, 2, 11
    m, wt = handle(E, H, I, K, act="gelu_tanh"), make(E, H, I)
    x, idx, w = tokens(n, H, E, K)
    bias = torch.randn((n, H), device="cuda").bfloat16()
    check(m, x, idx, w, wt, act="gelu_tanh", bias=bias, dtype=dtype)
    if dtype == torch.bfloat16:                     # the bias' own buffer as the output
        a = check(m, x, idx, w, wt, act="gelu_tanh", bias=bias)
        m.forward(x, idx, w, wt, bias, bias=bias)
        assert torch.equal(a, bias)


@pytest.mark.parametrize("weights,group", FORMS)
def test_equal_bits_on_repeats_streams_and_graphs(weights, group):
    E, H, I, K, n = 24, 1024, 384, 6, 37
    m, wt = handle(E, H, I, K, weights, group), make(E, H, I, weights, group)
    x, idx, w = tokens(n, H, E, K)
    a = torch.empty_like(x)
    m.forward(x, idx, w, wt, a)
    b = torch.empty_like(x)
    for _ in range(50):
        m.forward(x, idx, w, wt, b)
        assert torch.equal(a, b)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    m.forward(x, idx, w, wt, b.zero_(), stream=st)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.forward(x, idx, w, wt, b)
    for seed in range(5):
        x2, idx2, w2 = tokens(n, H, E, K, seed=seed + 100)
        x.copy_(x2), idx.copy_(idx2), w.copy_(w2)
        g.replay()
        m.forward(x, idx, w, wt, a)
        torch.cuda.synchronize()
        assert torch.equal(a, b)
    assert m.status() == 0


@pytest.mark.parametrize("weights,group", FORMS)
def test_layer_is_route_then_forward(weights, group):
    E, H, I, K, n = 16, 256, 128, 4, 13
    m, wt = handle(E, H, I, K, weights, group), make(E, H, I, weights, group)
    x, _, _ = tokens(n, H, E, K)
    z = torch.randn((n, E), device="cuda")
    z[2, 2:] = float("-inf")                        # two experts left
    z[5] = float("-inf")                            # none
    rc = ep.make_route_cfg(E, K, "softmax", True)
    idx, w = torch.empty((n, K), dtype=torch.int64, device="cuda"), torch.empty((n, K), device="cuda")
    i2, w2 = torch.empty_like(idx), torch.empty_like(w)
    a, b = torch.empty_like(x), torch.empty_like(x)
    m.layer(rc, x, z, wt, idx, w, a)
    ep.ep_route(rc, z, i2, w2)
    m.forward(x, i2, w2, wt, b)
    assert torch.equal(idx, i2) and torch.equal(w, w2) and torch.equal(a, b)
    assert (a[5] == 0).all() and m.status() == 0
    ref, tol = reference(x, idx, w, wt)
    assert ((a.double() - ref).abs() <= tol + 2.0 ** -7.99 * ref.abs()).all()


# the layer routes a few tokens in its own launch; whatever it does, it gives the router's bits
LAYERS = [(1, 1, 1), (1, 64, 8), (8, 256, 8), (8, 250, 7), (3, 33, 2), (5, 8, 8), (2, 31, 5), (8, 128, 6),
          (9, 64, 8), (8, 257, 4), (4, 40, 9), (8, 300, 16), (64, 256, 8), (33, 17, 3)]


@pytest.mark.parametrize("n,E,K", LAYERS)
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("sigmoid", True), ("sigmoid", False), ("softmax", False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_gives_the_bits_of_route_and_forward(n, E, K, score, renorm, dtype):
    H, I = 64, 32
    m, wt = handle(E, H, I, K), make(E, H, I)
    x, _, _ = tokens(n, H, E, K)
    g = torch.Generator(device="cuda").manual_seed(n * 1000 + E)
    wide = torch.randn((n, E + 3), device="cuda", generator=g)
    wide[torch.rand((n, E + 3), device="cuda", generator=g) < 0.2] = float("-inf")
    if n > 1:
        wide[1] = float("-inf")                     # nothing left
        wide[n - 1] = (2 * wide[n - 1]).round() / 2  # many equal scores
    z = wide.to(dtype)[:, 2:2 + E]                  # strided, not 16-byte aligned
    rc = ep.make_route_cfg(E, K, score, renorm, 1.5)
    idx = torch.full((n, K), -9, dtype=torch.int64, device="cuda")
    w = torch.full((n, K), float("nan"), device="cuda")
    i2, w2 = torch.empty_like(idx), torch.empty_like(w)
    a, b = torch.empty_like(x), torch.empty_like(x)
    for bias in (None, torch.linspace(-0.1, 0.1, E, device="cuda")):
        m.layer(rc, x, z, wt, idx, w, a, select_bias=bias)
        ep.ep_route(rc, z, i2, w2, bias)
        m.forward(x, i2, w2, wt, b)
        assert torch.equal(idx, i2) and torch.equal(w, w2) and torch.equal(a, b) and m.status() == 0


def test_agrees_with_layout_dispatch_experts_combine():
    # the same tokens through the framework's large-batch path, the experts in torch
    E, H, I, K, n = 32, 1024, 256, 4, 64
    wt = make(E, H, I)
    x, idx, w = tokens(n, H, E, K)
    m = handle(E, H, I, K)
    a = torch.empty_like(x)
    m.forward(x, idx, w, wt, a)
    hd = ep.EpHandle(ep.make_cfg(4, H, 32, 8, K))
    hd.layout(idx)
    recv = torch.zeros((hd.recv_capacity, H), dtype=torch.bfloat16, device="cuda")
    hd.dispatch(x, recv)
    y = torch.zeros_like(recv)
    psum = hd.field(ep.FIELD_PSUM_PER_EXPERT).tolist()
    for e in range(E):
        r = slice(psum[e], psum[e + 1])
        u = recv[r].double() @ wt.tensors[0][e].double().T
        y[r] = ((act64(u[:, :I], "silu") * u[:, I:]) @ wt.tensors[1][e].double().T).bfloat16()
    b = torch.empty_like(x)
    hd.combine(y, w, b)
    hd.free()
    # y's own rounding, 2^-9 of each expert row, on top of the tolerance of both
    ref, tol = reference(x, idx, w, wt)
    assert ((a.double() - b.double()).abs() <= 2 * tol + 2.0 ** -7 * w.sum(1, keepdim=True) * ref.abs().amax()).all()


def test_two_handles_on_two_streams():
    E, H, I, K, n = 16, 512, 512, 4, 8
    wt = make(E, H, I)
    ms = [handle(E, H, I, K) for _ in range(2)]
    data = [tokens(n, H, E, K, seed=s) for s in (1, 2)]
    want = [check(m, *d, wt) for m, d in zip(ms, data)]
    sts = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(d[0]) for d in data]
    torch.cuda.synchronize()
    for _ in range(40):
        for m, d, s, o in zip(ms, data, sts, outs):
            m.forward(*d, wt, o, stream=s)
    torch.cuda.synchronize()
    for o, r, m in zip(outs, want, ms):
        assert torch.equal(o, r) and m.status() == 0


def test_offsets_past_32_bits():
    # 2.4e9 elements in w13: the last experts lie past 2^32 bytes and 2^31 elements
    E, H, I, K, n = 140, 4096, 2104, 2, 3
    w13 = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros((E, H, I), dtype=torch.bfloat16, device="cuda")
    small = make(2, H, I)
    for at, e in ((0, 0), (1, E - 1)):
        w13[e].copy_(small.tensors[0][at])
        w2[e].copy_(small.tensors[1][at])
    x, _, w = tokens(n, H, 2, K)
    idx = torch.tensor([[0, E - 1], [E - 1, 0], [E - 1, -1]], device="cuda")
    m = handle(E, H, I, K, max_tokens=n)
    out = torch.empty_like(x)
    m.forward(x, idx, w, ep.EpMoeWeights(w13, w2), out)
    near = torch.where(idx == E - 1, 1, idx)
    ref, tol = reference(x, near, w, small)
    assert ((out.double() - ref).abs() <= tol + 2.0 ** -7.99 * ref.abs()).all()


def test_a_wait_that_gives_up_is_reported_and_leaves_the_next_call_sound(monkeypatch):
    # blocks wait for one another's rounds; with no time to wait at all some give up, go on
    # in bounds and report it.  Another handle, with time, is not affected.
    E, H, I, K, n = 64, 2048, 512, 8, 8
    wt = make(E, H, I)
    x, idx, w = tokens(n, H, E, K)
    good = handle(E, H, I, K)
    want = check(good, x, idx, w, wt)
    monkeypatch.setenv("EP_GB300_WAIT_NS", "0")
    m = handle(E, H, I, K)
    monkeypatch.delenv("EP_GB300_WAIT_NS")
    out = torch.empty_like(x)
    for _ in range(3):
        m.forward(x, idx, w, wt, out)
        assert m.status() == 2 and m.status() == 0
    good.forward(x, idx, w, wt, out)
    assert good.status() == 0 and torch.equal(out, want)
