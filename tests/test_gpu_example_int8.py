"""The example of an MoE block with int8 experts and the router's losses: it runs, and its
gradients are autograd's.

The output against unquantised experts: a row's rounding is uniform in a step of amax/127 (rms 0.29
steps), a normal row's amax is under 6 deviations, so each of the five 8-bit factors (x, the two
halves of w13, h, w2) is off by at most 1.4% rms; 4% together with the two roundings to bf16.  Losses and
gradient: fp32 sums, 2^-15 of their terms (the balance gradient's terms cancel against each other,
but the router's own gradient beside them does not)."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,sizes", [(1000, {}), (1, dict(sequences=1)),
                                          (77, dict(sequences=5, hidden=256, inter=208, experts=60, topk=6)),
                                          (3000, dict(sequences=2, hidden=512, inter=256, experts=8, topk=2))])
def test_int8_block(tokens, sizes):
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    sys.path.insert(0, os.path.join(__graft_entry__.ROOT, "examples"))
    import moe_int8
    out, losses, grad = moe_int8.main(tokens, **sizes)
    assert out < 0.04 and losses < 2.0 ** -15 and grad < 2.0 ** -14
