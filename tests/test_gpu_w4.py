"""Products with 4-bit weights against a plain implementation in 64 bits.

Two kinds of inputs.  Whole numbers with scales that are powers of two: every
product and partial sum is exact in fp32 whatever the order, so fp32 outputs have
to be equal and bf16 outputs have to be the exact sum's rounding.  Random ones:
at most cols/16 + 32 additions in a chain, each off by 2^-23 of the sum S of
absolute products (matrix instructions may truncate), so (cols/16 + 32) 2^-23 S,
and for bf16 the rounding of 2^-8 of the value (8 significant
bits).
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
    rows, half = q.shape
    w = torch.empty((rows, 2 * half), dtype=torch.float64, device=q.device)
    w[:, 0::2] = (q & 15).double() - 8
    w[:, 1::2] = (q >> 4).double() - 8
    return w * s.double().repeat_interleave(2 * half // s.shape[1], 1)


def make(n, rows, cols, group, whole, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + n * 131 + rows * 17 + cols)
    q = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device="cuda", generator=g)
    if whole:
        x = torch.randint(-3, 4, (n, cols), device="cuda", generator=g).bfloat16()
        s = 2.0 ** torch.randint(-2, 2, (rows, cols // group), device="cuda", generator=g).float()
    else:
        x = torch.randn((n, cols), device="cuda", generator=g).bfloat16()
        s = torch.rand((rows, cols // group), device="cuda", generator=g) + 0.1
    return x, q, s


def check(x, q, s, dtype, whole):
    out = torch.full((x.shape[0], q.shape[0]), float("nan"), dtype=dtype, device="cuda")
    ep.ep_w4_linear(x, q, s, out)
    w = dense(q, s)
    ref = x.double() @ w.T
    if whole:
        assert torch.equal(out, ref.to(dtype))
        return
    bound = (x.shape[1] / 16 + 32) * 2.0 ** -23 * (x.double().abs() @ w.abs().T)
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -7.99 * ref.abs()
    assert ((out.double() - ref).abs() <= bound).all()


SIZES = [(1, 1, 32, 32), (1, 16, 64, 64), (2, 17, 96, 32), (3, 15, 128, 128), (1, 1024, 1024, 32),
         (5, 63, 320, 64), (7, 64, 384, 128), (8, 65, 160, 32), (9, 130, 256, 64), (16, 257, 640, 128),
         (17, 100, 1056, 32), (24, 31, 2048, 128), (25, 33, 512, 64), (33, 200, 1152, 128),
         (48, 48, 224, 32), (63, 129, 448, 64), (64, 500, 4096, 128), (1, 4099, 2112, 64),
         (4, 2000, 7168, 128), (32, 777, 5120, 32), (1, 40, 14336, 128)]


@pytest.mark.parametrize("n,rows,cols,group", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_whole_numbers_are_exact(n, rows, cols, group, dtype):
    check(*make(n, rows, cols, group, True), dtype, True)


@pytest.mark.parametrize("n,rows,cols,group", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_random_values(n, rows, cols, group, dtype):
    check(*make(n, rows, cols, group, False), dtype, False)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_every_number_of_tokens(group):
    x, q, s = make(64, 96, 384, group, True)
    for n in range(65):
        check(x[:n].contiguous(), q, s, torch.float32, True)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_each_nibble_and_column_in_its_place(group):
    # x picks one column at a time: the output is that column of the matrix
    cols = 2 * group
    _, q, s = make(1, 40, cols, group, True)
    w = dense(q, s)
    for c0 in range(0, cols, 64):
        m = min(64, cols - c0)
        x = torch.zeros((m, cols), device="cuda")
        x[torch.arange(m), c0 + torch.arange(m)] = 1.0
        out = torch.empty((m, 40), device="cuda")
        ep.ep_w4_linear(x.bfloat16(), q, s, out)
        assert torch.equal(out.double(), w[:, c0:c0 + m].T)


def test_a_token_of_nan_or_infinity_stays_its_own():
    x, q, s = make(11, 100, 512, 64, True)
    out = torch.empty((11, 100), device="cuda")
    ep.ep_w4_linear(x, q, s, out)
    bad = x.clone()
    bad[3] = float("nan")
    bad[7, 100] = float("inf")
    got = torch.empty_like(out)
    ep.ep_w4_linear(bad, q, s, got)
    keep = [t for t in range(11) if t not in (3, 7)]
    assert torch.equal(got[keep], out[keep])
    assert got[3].isnan().all()
    # 0 * inf is NaN, the others are infinite
    w = dense(q, s)[:, 100]
    assert got[7][w == 0].isnan().all() and torch.equal(got[7][w > 0], torch.full_like(got[7][w > 0], float("inf")))


@pytest.mark.parametrize("n", [1, 3, 8, 11, 33, 64])
def test_huge_activations_are_exact_and_infinite_ones_keep_their_sign(n):
    # all of a token times 2^70; an infinite column in another token
    x, q, s = make(n, 100, 512, 64, True)
    big = x.clone()
    big[n // 2] *= 2.0 ** 70
    check(big, q, s, torch.float32, True)
    big[0] = 0.0
    big[0, 77] = -float("inf")
    out = torch.empty((n, 100), device="cuda")
    ep.ep_w4_linear(big, q, s, out)
    w = dense(q, s)[:, 77]
    assert out[0][w == 0].isnan().all()
    assert (out[0][w > 0] == -float("inf")).all() and (out[0][w < 0] == float("inf")).all()


@pytest.mark.parametrize("n", [1, 3, 8, 11, 33, 64])
def test_tiny_activations_are_exact(n):
    x, q, s = make(n, 100, 512, 64, True)
    x[::2] *= 2.0 ** -80
    check(x, q, s, torch.float32, True)


def test_scales_of_zero_and_negative_scales():
    x, q, s = make(4, 64, 256, 64, True)
    s[::3] = 0.0
    s[1::3] *= -1.0
    check(x, q, s, torch.float32, True)


def test_nothing_outside_the_output_is_written():
    x, q, s = make(6, 37, 128, 64, True)
    buf = torch.full((6 * 37 + 64,), 5.0, device="cuda")
    ep.ep_w4_linear(x, q, s, buf[32:32 + 6 * 37].view(6, 37))
    assert (buf[:32] == 5.0).all() and (buf[32 + 6 * 37:] == 5.0).all()
    b16 = torch.full((6 * 37 + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_w4_linear(x, q, s, b16[33:33 + 6 * 37].view(6, 37))
    assert (b16[:33] == 5.0).all() and (b16[33 + 6 * 37:] == 5.0).all()


def test_equal_bits_and_other_stream_and_graph():
    x, q, s = make(19, 640, 1536, 128, False)
    a = torch.empty((19, 640), device="cuda")
    ep.ep_w4_linear(x, q, s, a)
    b = torch.empty_like(a)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    ep.ep_w4_linear(x, q, s, b, stream=st)
    st.synchronize()
    assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ep.ep_w4_linear(x, q, s, b)
    x.copy_(torch.randn((19, 1536), device="cuda").bfloat16())
    g.replay()
    ep.ep_w4_linear(x, q, s, a)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_more_than_2_31_weights():
    # 2^31 + columns of packed weights: offsets pass 32 bits
    rows, cols = 300000, 14336
    q = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device="cuda")
    s = torch.full((rows, cols // 128), 0.5, device="cuda")
    x = torch.randint(-1, 2, (2, cols), device="cuda").bfloat16()
    out = torch.empty((2, rows), device="cuda")
    ep.ep_w4_linear(x, q, s, out)
    pick = torch.cat((torch.arange(64), torch.arange(149990, 150010), torch.arange(rows - 64, rows))).cuda()
    assert torch.equal(out[:, pick].double(), x.double() @ dense(q[pick], s[pick]).T)
