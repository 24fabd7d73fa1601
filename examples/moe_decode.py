"""One decode step of an MoE block with 4-bit weights, through the package's entry points:
the router's top-k, the chosen experts' gated products and their weighted sum (EpMoe.layer),
and a shared expert of two 4-bit projections (ep_w4_linear) that enters as the layer's bias.
The step is captured once and replayed as a CUDA graph.

    python examples/moe_decode.py [tokens]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_ep_layout_gb300 as ep  # noqa: E402


def quantize(w, group):
    """bf16 or fp32 weights [..., rows, cols] to the 4-bit form: packed nibbles and fp32 scales."""
    w = w.float().unflatten(-1, (-1, group))
    scales = w.abs().amax(-1) / 7.0
    q = torch.where(scales[..., None] > 0, w / scales[..., None], 0.0).round().clamp(-8, 7).to(torch.int16) + 8
    q = q.flatten(-2).to(torch.uint8)
    return (q[..., 0::2] | (q[..., 1::2] << 4)).contiguous(), scales.contiguous()


def dequantize(q, scales):
    v = torch.stack((q & 15, q >> 4), -1).float().flatten(-2) - 8.0
    return (v.unflatten(-1, (scales.shape[-1], -1)) * scales[..., None]).flatten(-2)


class Block:
    def __init__(self, hidden=1024, inter=512, experts=32, topk=4, group=128, max_tokens=16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return torch.randn(shape, device="cuda", generator=g) * shape[-1] ** -0.5
        self.hidden, self.inter, self.experts, self.topk = hidden, inter, experts, topk
        self.gate = weight(experts, hidden)
        self.w13, self.s13 = quantize(weight(experts, 2 * inter, hidden), group)
        self.w2, self.s2 = quantize(weight(experts, hidden, inter), group)
        self.shared13 = quantize(weight(2 * inter, hidden), group)
        self.shared2 = quantize(weight(hidden, inter), group)
        self.route = ep.make_route_cfg(experts, topk, "sigmoid", renormalize=True, scale=2.5)
        self.moe = ep.EpMoe(ep.make_moe_cfg(hidden, inter, experts, topk, max_tokens, "int4", group))
        self.weights = ep.EpMoeWeights(self.w13, self.w2, self.s13, self.s2)

    def buffers(self, n):
        def new(*s, dtype=torch.bfloat16):
            return torch.empty(s, dtype=dtype, device="cuda")
        return dict(x=new(n, self.hidden), idx=new(n, self.topk, dtype=torch.int64),
                    w=new(n, self.topk, dtype=torch.float32), up=new(n, 2 * self.inter, dtype=torch.float32),
                    shared=new(n, self.hidden), out=new(n, self.hidden))

    def step(self, b):
        """out = sum over the chosen experts + the shared expert, for the tokens in b["x"]."""
        x = b["x"]
        logits = x.float() @ self.gate.T
        ep.ep_w4_linear(x, *self.shared13, b["up"])
        h = (torch.nn.functional.silu(b["up"][:, :self.inter]) * b["up"][:, self.inter:]).bfloat16()
        ep.ep_w4_linear(h, *self.shared2, b["shared"])
        self.moe.layer(self.route, x, logits, self.weights, b["idx"], b["w"], b["out"], bias=b["shared"])

    def reference(self, b):
        """The same in plain torch, with the experts that the step chose."""
        x = b["x"].float()

        def expert(x, w13, w2):
            u = x @ w13.T
            return (torch.nn.functional.silu(u[:, :self.inter]) * u[:, self.inter:]) @ w2.T
        y = expert(x, dequantize(*self.shared13), dequantize(*self.shared2))
        for t in range(x.shape[0]):
            for e, w in zip(b["idx"][t].tolist(), b["w"][t].tolist()):
                y[t] += w * expert(x[t:t + 1], dequantize(self.w13[e], self.s13[e]),
                                   dequantize(self.w2[e], self.s2[e]))[0]
        return y


def main(tokens=8, **sizes):
    block = Block(max_tokens=tokens, **sizes)
    b = block.buffers(tokens)
    b["x"].normal_()
    block.step(b)                                   # once outside the graph: kernels are set up
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step(b)
    b["x"].normal_()
    graph.replay()
    ref = block.reference(b)
    err = ((b["out"].float() - ref).norm() / ref.norm()).item()
    assert block.moe.status() == 0
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(100):
        graph.replay()
    end.record()
    end.synchronize()
    print("%d tokens: %.1f us a step, off the plain form by %.1e" % (tokens, start.elapsed_time(end) * 10, err))
    return err


if __name__ == "__main__":
    main(*[int(a) for a in sys.argv[1:2]])
