"""How many bits of h, the gated product between an expert's two matrices, reach the output:
16 with a bf16 output, all 24 with an fp32 one.

Exact inputs: gates of 64 (silu(64) is 64 in fp32) and up projections that are whole numbers
of 14 bits (20 bits: 2^19 + 2^11 and a low end, three bf16) with a low end that differs from
token to token, entry to entry and channel to channel; a down weight of one channel, or the difference of two, so that the sums
are exact in fp32 and the low ends are what is left of them.  The output has to be equal.

Random inputs, fp32 output: the 2-norm of the error against 64 bits, relative to the
output's.  A matrix instruction may truncate a sum of 16 products, 2^-23 of it; a warp adds
cols/128 of them and 8 warps' sums: independent errors of 2^-23 sqrt(cols/128 + 8), for 2048
and 1024 columns 2^-20.7 and 2^-21.0; with the gate and the up projection of h 2^-20.2 and
together 2^-19.8; exp adds 2^-22.  The bound is 2^-19.5; h in 16 bits alone is off by
2^-17 / sqrt(3) at the most and 2^-18.6 in the mean over a binade.
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


def pack(v, group, scale):
    """Whole numbers from -8 to 7 [..., rows, cols] to the 4-bit form with one scale for a row."""
    q = (v + 8).to(torch.uint8)
    s = scale[..., None].expand(*v.shape[:-1], v.shape[-1] // group)
    return (q[..., 0::2] | q[..., 1::2] << 4).contiguous(), s.contiguous()


def exact_case(E, H, I, big, form, group, seed):
    """x column 0 is 1 (the gate reads it), columns 1 and 8 are big, 2..7 are small; w2's even
    rows take one channel, its odd rows the difference of two."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w13 = torch.zeros((E, 2 * I, H), device="cuda")
    w13[:, :I, 0] = 4.0
    w13[:, I:, [1, 8]] = 1.0
    w13[:, I:, 2:8] = torch.randint(-3, 4, (E, I, 6), device="cuda", generator=g).float()
    w2 = torch.zeros((E, H, I), device="cuda")
    r = torch.arange(H, device="cuda")
    for e in range(E):
        w2[e, r, (r * 7 + e) % I] = 1.0
        odd = r[1::2]
        w2[e, odd, (odd * 7 + e + 1 + odd % (I - 1)) % I] = -1.0
    gate = torch.full((E, 2 * I), 1.0, device="cuda")
    gate[:, :I] = 16.0
    if form == "bf16":
        wt = ep.EpMoeWeights((w13 * gate[..., None]).bfloat16(), w2.bfloat16())
    else:
        (q13, s13), (q2, s2) = pack(w13, group, gate), pack(w2, group, torch.ones((E, H), device="cuda"))
        wt = ep.EpMoeWeights(q13, q2, s13, s2)

    def tokens(n, K):
        x = torch.zeros((n, H), device="cuda")
        x[:, 0] = 1.0
        x[:, 1], x[:, 8] = big
        x[:, 2:8] = torch.randint(-5, 6, (n, 6), device="cuda", generator=g).float()
        idx = torch.rand((n, E), device="cuda", generator=g).argsort(1)[:, :K].contiguous()
        return x, idx
    return wt, tokens, w13 * gate[..., None], w2


CASES = [("bf16", 0, n) for n in (1, 3, 4, 5, 17, 64)] + [("int4", 64, n) for n in (1, 4, 8, 9, 64)] + \
        [("int4", 32, 8), ("int4", 128, 40)]


@pytest.mark.parametrize("form,group,n", CASES)
@pytest.mark.parametrize("E,K", [(1, 1), (5, 2), (16, 4)])
@pytest.mark.parametrize("dtype,big", [(torch.bfloat16, (2.0 ** 13, 0.0)), (torch.float32, (2.0 ** 13, 0.0)),
                                       (torch.float32, (2.0 ** 19, 2.0 ** 11))])
def test_low_bits_of_h_arrive(form, group, n, E, K, dtype, big):
    H, I = 256, 128
    wt, tokens, w13, w2 = exact_case(E, H, I, big, form, group, seed=n + E)
    x, idx = tokens(n, K)
    w = torch.ones((n, K), device="cuda")
    m = ep.EpMoe(ep.make_moe_cfg(H, I, E, K, 64, form, group))
    out = torch.full((n, H), float("nan"), dtype=dtype, device="cuda")
    m.forward(x.bfloat16(), idx, w, wt, out)
    want = torch.zeros((n, H), dtype=torch.float64, device="cuda")
    for t in range(n):
        for e in idx[t].tolist():
            u = w13[e].double() @ x[t].double()
            want[t] += w2[e].double() @ (u[:I] * u[I:])
    assert torch.equal(out, want.to(dtype)) and m.status() == 0


@pytest.mark.parametrize("form,group", [("bf16", 0), ("int4", 32), ("int4", 128)])
@pytest.mark.parametrize("n,E,K", [(1, 4, 2), (4, 4, 2), (8, 8, 8), (13, 6, 3), (64, 8, 4)])
def test_fp32_output_is_as_exact_as_fp32(form, group, n, E, K):
    H, I = 2048, 1024
    g = torch.Generator(device="cuda").manual_seed(n)

    def one(rows, cols):
        if form == "bf16":
            return (torch.randn((E, rows, cols), device="cuda", generator=g) * cols ** -0.5).bfloat16(), None
        q = torch.randint(0, 256, (E, rows, cols // 2), dtype=torch.uint8, device="cuda", generator=g)
        return q, (torch.rand((E, rows, cols // group), device="cuda", generator=g) + 0.5) / (4.6 * cols ** 0.5)

    def dense(q, s):
        if s is None:
            return q.double()
        v = torch.stack((q & 15, q >> 4), -1).flatten(-2).double() - 8
        return v * s.double().repeat_interleave(group, -1)
    w13, s13 = one(2 * I, H)
    w2, s2 = one(H, I)
    x = torch.randn((n, H), device="cuda", generator=g).bfloat16()
    idx = torch.rand((n, E), device="cuda", generator=g).argsort(1)[:, :K].contiguous()
    w = torch.rand((n, K), device="cuda", generator=g)
    m = ep.EpMoe(ep.make_moe_cfg(H, I, E, K, 64, form, group))
    out = torch.empty((n, H), device="cuda")
    m.forward(x, idx, w, ep.EpMoeWeights(w13, w2, s13, s2), out)
    want = torch.zeros((n, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, k = (idx == e).nonzero(as_tuple=True)
        u = x[t].double() @ dense(w13[e], None if s13 is None else s13[e]).T
        h = u[:, :I] * torch.sigmoid(u[:, :I]) * u[:, I:]
        want.index_add_(0, t, w[t, k].double()[:, None] * (h @ dense(w2[e], None if s2 is None else s2[e]).T))
    assert ((out.double() - want).norm() / want.norm()).item() < 2.0 ** -19.5 and m.status() == 0
