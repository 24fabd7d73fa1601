"""The example of a decode step: router, 4-bit experts, 4-bit shared expert as the bias.

Against plain fp32 torch: the shared expert's h and output and the result are each rounded
to bf16 (2^-8 of a value at most, under 2^-9 rms), so the 2-norm of the difference stays
below 2^-7 of the result's."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,sizes", [(1, {}), (8, {}), (13, dict(hidden=512, inter=384, experts=60, topk=6, group=64)),
                                          (64, dict(hidden=256, inter=160, experts=8, topk=2, group=32))])
def test_decode_step(tokens, sizes):
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    sys.path.insert(0, os.path.join(__graft_entry__.ROOT, "examples"))
    import moe_decode
    assert moe_decode.main(tokens, **sizes) < 2.0 ** -7
