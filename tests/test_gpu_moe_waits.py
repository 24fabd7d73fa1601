"""The MoE layer's bounded waits: every way out, taken at once with a limit of 0 (a warp that
waits for another one of its block, or for another block, gives up at its first test), and
limits so long that no sum of them may wrap.  Results of a call that gave up are not looked
at: it has to end, to be reported, and to leave everything beside its own output alone.
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


def weights(E, H, I, form, group):
    g = torch.Generator(device="cuda").manual_seed(H + I)

    def one(rows, cols):
        if form == "bf16":
            return (torch.randn((E, rows, cols), device="cuda", generator=g) * cols ** -0.5).bfloat16(), None
        q = torch.randint(0, 256, (E, rows, cols // 2), dtype=torch.uint8, device="cuda", generator=g)
        return q, torch.rand((E, rows, cols // group), device="cuda", generator=g) / cols ** 0.5
    w13, s13 = one(2 * I, H)
    w2, s2 = one(H, I)
    return ep.EpMoeWeights(w13, w2, s13, s2)


def inputs(n, H, E, K):
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn((n, H), device="cuda", generator=g).bfloat16()
    idx = torch.rand((n, E), device="cuda", generator=g).argsort(1)[:, :K].contiguous()
    return x, idx, torch.rand((n, K), device="cuda", generator=g)


def handle(monkeypatch, wait_ns, E, H, I, K, form, group):
    if wait_ns is not None:
        monkeypatch.setenv("EP_GB300_WAIT_NS", str(wait_ns))
    m = ep.EpMoe(ep.make_moe_cfg(H, I, E, K, 64, form, group))
    monkeypatch.delenv("EP_GB300_WAIT_NS", raising=False)
    return m


# the last ones have blocks with more than the 64 rounds that may be written and not told
SHAPES = [(1, 1, 1, 64, 64), (3, 2, 8, 256, 128), (8, 8, 64, 2048, 512), (64, 8, 64, 1024, 512),
          (64, 8, 16, 8192, 4096)]


@pytest.mark.parametrize("form,group", [("bf16", 0), ("int4", 32), ("int4", 128)])
@pytest.mark.parametrize("n,K,E,H,I", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_limit_of_nothing(monkeypatch, n, K, E, H, I, form, group, dtype):
    if group > min(H, I):
        group = 32
    wt = weights(E, H, I, form, group)
    x, idx, w = inputs(n, H, E, K)
    sound = handle(monkeypatch, None, E, H, I, K, form, group)
    want = torch.empty((n, H), dtype=dtype, device="cuda")
    sound.forward(x, idx, w, wt, want)
    assert sound.status() == 0
    m = handle(monkeypatch, 0, E, H, I, K, form, group)
    guarded = torch.full((n + 2, H), 7.0, dtype=dtype, device="cuda")
    for _ in range(5):
        m.forward(x, idx, w, wt, guarded[1:n + 1])
    assert m.status() == 2 and m.status() == 0
    assert (guarded[0] == 7.0).all() and (guarded[-1] == 7.0).all()
    # nothing to wait for: no entry is left
    m.forward(x, torch.full_like(idx, -1), w, wt, guarded[1:n + 1])
    assert m.status() == 0 and (guarded[1:n + 1] == 0).all()
    got = torch.empty_like(want)
    sound.forward(x, idx, w, wt, got)
    assert sound.status() == 0 and torch.equal(got, want)


@pytest.mark.parametrize("wait_ns", [3 * 10 ** 9, 2 ** 63, 2 ** 64 - 1])
def test_limits_longer_than_the_wait_inside_a_block(monkeypatch, wait_ns):
    E, H, I, K, n = 16, 1024, 512, 4, 20
    wt = weights(E, H, I, "bf16", 0)
    x, idx, w = inputs(n, H, E, K)
    want, got = torch.empty_like(x), torch.empty_like(x)
    handle(monkeypatch, None, E, H, I, K, "bf16", 0).forward(x, idx, w, wt, want)
    m = handle(monkeypatch, wait_ns, E, H, I, K, "bf16", 0)
    for _ in range(3):
        m.forward(x, idx, w, wt, got)
        assert m.status() == 0 and torch.equal(got, want)
