"""4-bit weights at the ends of the range, for few tokens and for more: what the products
lose does not depend on how large or small activations and scales are, on the weights that
are zero, nor on the number of tokens.

Exact inputs: one weight of a row is not zero, so that the output is one product of 8, 4
and a power of two's bits.  Scaling: x, or the scales, times a power of two gives the same
output bits times it, as long as nothing leaves fp32's normal numbers.  Random inputs as in
test_gpu_w4: at most cols/16 + 32 additions in a chain, each off by 2^-23 of the sum of
absolute products.
"""
import pytest
import torch

import combine_ep_layout_gb300 as ep

pytestmark = pytest.mark.gpu

TOKENS = [1, 3, 8, 9, 16, 33, 64]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def dense(q, s):
    w = torch.stack((q & 15, q >> 4), -1).flatten(-2).double() - 8
    return w * s.double().repeat_interleave(w.shape[-1] // s.shape[-1], -1)


def make(n, rows, cols, group):
    g = torch.Generator(device="cuda").manual_seed(n + rows + cols + group)
    x = torch.randn((n, cols), device="cuda", generator=g).bfloat16()
    q = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.rand((rows, cols // group), device="cuda", generator=g) + 0.1
    return x, q, s


def linear(x, q, s):
    out = torch.full((x.shape[0], q.shape[0]), float("nan"), device="cuda")
    ep.ep_w4_linear(x, q, s, out)
    return out


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n", TOKENS)
def test_zero_weights_take_no_bits(n, group):
    rows, cols = 150, 768
    x, q, s = make(n, rows, cols, group)
    x = (x.abs() + 1.0).bfloat16()
    w = torch.full((rows, cols), 8, dtype=torch.uint8, device="cuda")
    r = torch.arange(rows, device="cuda")
    w[r, (r * 5) % cols] = (r % 16).to(torch.uint8)
    q = w[:, 0::2] | w[:, 1::2] << 4
    s = 2.0 ** torch.randint(-3, 3, s.shape, device="cuda").float()
    assert torch.equal(linear(x, q, s).double(), x.double() @ dense(q, s).T)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n", TOKENS)
@pytest.mark.parametrize("up", [-90, -50, 30, 60, 90])
def test_scaled_activations_give_the_same_bits(n, group, up):
    x, q, s = make(n, 150, 768, group)
    assert torch.equal(linear(x * 2.0 ** up, q, s), linear(x, q, s) * 2.0 ** up)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n", TOKENS)
@pytest.mark.parametrize("up", [-90, 90])
def test_scaled_scales_give_the_same_bits(n, group, up):
    x, q, s = make(n, 150, 768, group)
    assert torch.equal(linear(x, q, s * 2.0 ** up), linear(x, q, s) * 2.0 ** up)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n", TOKENS)
@pytest.mark.parametrize("x_by,s_by", [(-80, -30), (-100, -10), (-128, 100)])   # the last: bf16's subnormals
def test_tiny_activations_and_scales(n, group, x_by, s_by):
    x, q, s = make(n, 150, 768, group)
    x, s = x * 2.0 ** x_by, s * 2.0 ** s_by
    w = dense(q, s)
    bound = (x.shape[1] / 16 + 32) * 2.0 ** -23 * (x.double().abs() @ w.abs().T)
    assert ((linear(x, q, s).double() - x.double() @ w.T).abs() <= bound).all()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n", TOKENS)
def test_an_infinite_activation_reaches_its_own_products(n, group):
    x, q, s = make(n, 150, 768, group)
    x[0, 100] = float("inf")
    w = dense(q, s)[:, 100]
    out = linear(x, q, s)
    assert out[0][w == 0].isnan().all()
    assert (out[0][w > 0] == float("inf")).all() and (out[0][w < 0] == -float("inf")).all()
    assert torch.isfinite(out[1:]).all()


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("n", [1, 8, 9, 40])
@pytest.mark.parametrize("up", [-90, -60, 60, 90])
def test_moe_layer_scaled_up_projection_gives_the_same_bits(n, group, up):
    E, H, I, K = 6, 384, 256, 2
    g = torch.Generator(device="cuda").manual_seed(n)
    q13 = torch.randint(0, 256, (E, 2 * I, H // 2), dtype=torch.uint8, device="cuda", generator=g)
    q2 = torch.randint(0, 256, (E, H, I // 2), dtype=torch.uint8, device="cuda", generator=g)
    s13 = (torch.rand((E, 2 * I, H // group), device="cuda", generator=g) + 0.5) / (4.6 * H ** 0.5)
    s2 = (torch.rand((E, H, I // group), device="cuda", generator=g) + 0.5) / (4.6 * I ** 0.5)
    x = torch.randn((n, H), device="cuda", generator=g).bfloat16()
    idx = torch.rand((n, E), device="cuda", generator=g).argsort(1)[:, :K].contiguous()
    w = torch.rand((n, K), device="cuda", generator=g)
    m = ep.EpMoe(ep.make_moe_cfg(H, I, E, K, 64, "int4", group))
    a, b = (torch.empty((n, H), device="cuda") for _ in range(2))
    m.forward(x, idx, w, ep.EpMoeWeights(q13, q2, s13, s2), a)
    s13[:, I:] *= 2.0 ** up
    m.forward(x, idx, w, ep.EpMoeWeights(q13, q2, s13, s2), b)
    assert torch.equal(b, a * 2.0 ** up) and m.status() == 0
