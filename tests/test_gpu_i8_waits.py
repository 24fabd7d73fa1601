"""The int8 products' bounded waits: every way out, taken at once with a limit of 0 (a warp gives
up at its first test that fails), and limits of every length.  Results of a call that gave up are not
looked at: it has to end, to be reported, and to leave everything beside its own output alone."""
import pytest
import torch

import combine_ep_layout_gb300 as ep

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    assert ep.ep_i8_status() in (0, 2)


def call(n, rows, cols, act):
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randint(-127, 128, (n, cols), device="cuda", generator=g).to(torch.int8)
    w = torch.randint(-127, 128, (rows, cols), device="cuda", generator=g).to(torch.int8)
    xs, ws = torch.rand(n, device="cuda", generator=g), torch.rand(rows, device="cuda", generator=g)
    out = torch.full((n + 2, rows // 2 if act else rows), 7.0, dtype=torch.bfloat16, device="cuda")
    return out, lambda: ep.ep_i8_linear(x, xs, w, ws, out[1:n + 1], activation=act)


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("n,rows,cols", [(30, 64, 128), (60, 4096, 1024), (120, 1000, 4096), (300, 2048, 2048), (2000, 4096, 512)])
def test_a_limit_of_nothing(monkeypatch, n, rows, cols, act):
    out, run = call(n, rows, cols, act)
    run()
    assert ep.ep_i8_status() == 0
    want = out.clone()
    monkeypatch.setenv("EP_GB300_WAIT_NS", "0")
    for _ in range(5):
        run()
    assert ep.ep_i8_status() == 2 and ep.ep_i8_status() == 0
    assert (out[0] == 7.0).all() and (out[-1] == 7.0).all()
    monkeypatch.delenv("EP_GB300_WAIT_NS")
    run()
    assert ep.ep_i8_status() == 0 and torch.equal(out, want)


@pytest.mark.parametrize("wait_ns", [10 ** 9, 2 ** 63, 2 ** 64 - 1])
def test_long_limits(monkeypatch, wait_ns):
    out, run = call(200, 1024, 1024, "silu")
    run()
    want = out.clone()
    monkeypatch.setenv("EP_GB300_WAIT_NS", str(wait_ns))
    for _ in range(3):
        out.fill_(7.0)
        run()
        assert ep.ep_i8_status() == 0 and torch.equal(out, want)


def test_few_tokens_wait_for_nothing(monkeypatch):
    out, run = call(3, 512, 1024, None)
    run()
    want = out.clone()
    monkeypatch.setenv("EP_GB300_WAIT_NS", "0")
    run()
    assert ep.ep_i8_status() == 0 and torch.equal(out, want)
