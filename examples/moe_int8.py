"""An MoE block on a batch of sequences with int8 experts, through the package's entry points: the
router's top-k and its losses (EpBalance) with the gradient of the scores, and the experts between
dispatch and combine in 8 bits (ep_i8_dispatch, ep_i8_grouped, ep_i8_quantize).  The step is
captured once and replayed as a CUDA graph.

    python examples/moe_int8.py [tokens]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_ep_layout_gb300 as ep  # noqa: E402


def quantize(w):
    """bf16 or fp32 weights [experts, rows, cols] to int8 and a scale for each row."""
    q = torch.empty(w.shape, dtype=torch.int8, device=w.device)
    scales = torch.empty(w.shape[:2], dtype=torch.float32, device=w.device)
    ep.ep_i8_quantize(w.flatten(0, 1), q.flatten(0, 1), scales.flatten())
    return q, scales


class Block:
    def __init__(self, tokens, sequences=4, hidden=1024, inter=512, experts=32, topk=4, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return torch.randn(shape, device="cuda", generator=g) * shape[-1] ** -0.5

        def new(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device="cuda")
        f32, i8 = torch.float32, torch.int8
        self.inter, self.topk, self.experts = inter, topk, experts
        self.gate = weight(experts, hidden)
        self.w13, self.w2 = weight(experts, 2 * inter, hidden), weight(experts, hidden, inter)
        self.q13, self.s13 = quantize(self.w13)
        self.q2, self.s2 = quantize(self.w2)
        self.route = ep.make_route_cfg(experts, topk)
        self.balance = ep.EpBalance(self.route, tokens, sequences)
        self.handle = ep.EpHandle(ep.make_cfg(1, hidden, tokens, experts, topk, 16, "bf16", True))
        self.offsets = torch.linspace(0, tokens, sequences + 1).int().cuda()
        self.grad_loss = torch.tensor([0.01, 0.001], device="cuda")      # the losses' coefficients
        self.x, self.out, self.logits = new(tokens, hidden), new(tokens, hidden), new(tokens, experts, dtype=f32)
        self.idx, self.weights = new(tokens, topk, dtype=torch.int64), new(tokens, topk, dtype=f32)
        self.grad_weights, self.grad_logits = new(tokens, topk, dtype=f32), new(tokens, experts, dtype=f32)
        self.counts, self.sums = new(sequences, experts, dtype=torch.int32), new(sequences, experts, dtype=f32)
        self.tokens, self.loss = new(sequences + 1, dtype=torch.int32), new(2, dtype=f32)
        rows = self.handle.recv_capacity
        self.xq, self.xs = new(rows, hidden, dtype=i8), new(rows, dtype=f32)
        self.h, self.hq, self.hs = new(rows, inter), new(rows, inter, dtype=i8), new(rows, dtype=f32)
        self.y = new(rows, hidden)

    def step(self):
        """out = the experts' weighted sum; grad_logits = the router's gradient and the losses'."""
        torch.matmul(self.x.float(), self.gate.T, out=self.logits)
        ep.ep_route(self.route, self.logits, self.idx, self.weights)
        self.balance.forward(self.logits, self.idx, self.counts, self.sums, self.tokens, self.loss,
                             seq_offsets=self.offsets)
        self.handle.layout(self.idx)
        ep.ep_i8_dispatch(self.handle, self.x, self.xq, self.xs)
        ep.ep_i8_grouped(self.handle, self.xq, self.xs, self.q13, self.s13, self.h, activation="silu")
        ep.ep_i8_quantize(self.h, self.hq, self.hs, only_of=self.handle)
        ep.ep_i8_grouped(self.handle, self.hq, self.hs, self.q2, self.s2, self.y)
        self.handle.combine(self.y, self.weights, self.out)
        ep.ep_route_backward(self.route, self.logits, self.idx, self.grad_weights, self.grad_logits)
        self.balance.backward(self.logits, self.idx, self.counts, self.tokens, self.grad_loss, self.grad_logits,
                              seq_offsets=self.offsets, accumulate=True)

    def reference(self):
        """The same in plain torch with unquantised weights: out, the losses, and by autograd the gradient."""
        z = self.logits.double().requires_grad_()
        top = torch.gather(z, 1, self.idx)
        w = torch.softmax(top, 1)
        p = torch.softmax(z, 1)
        m, e, k = len(self.offsets) - 1, self.experts, self.topk
        loss = z.new_zeros(())
        for a, b in zip(self.offsets.tolist(), self.offsets.tolist()[1:]):
            if b > a:
                counts = torch.bincount(self.idx[a:b].flatten(), minlength=e).double()
                loss = loss + e / (k * m * (b - a) ** 2) * (counts * p[a:b].sum(0)).sum()
        losses = torch.stack([loss, torch.logsumexp(z, 1).square().mean()])
        ((w * self.grad_weights).sum() + (losses * self.grad_loss).sum()).backward()
        out = torch.zeros_like(self.x, dtype=torch.float32)
        for i in range(e):
            t, c = (self.idx == i).nonzero(as_tuple=True)
            u = self.x[t].float() @ self.w13[i].T
            u = torch.nn.functional.silu(u[:, :self.inter]) * u[:, self.inter:] @ self.w2[i].T
            out.index_add_(0, t, u * self.weights[t, c, None])
        return out, losses.detach(), z.grad


def main(tokens=1000, **sizes):
    block = Block(tokens, **sizes)
    block.x.normal_()
    block.grad_weights.normal_()
    block.step()                                    # once outside the graph: kernels are set up
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step()
    block.x.normal_()
    graph.replay()
    out, losses, grad = block.reference()
    assert block.handle.status() == 0 and ep.ep_i8_status() == 0
    errors = [((a - b).norm() / b.norm()).item() for a, b in
              ((block.out.float(), out), (block.loss.double(), losses), (block.grad_logits.double(), grad))]
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(100):
        graph.replay()
    end.record()
    end.synchronize()
    print("%d tokens: %.1f us a step; off plain torch: output %.1e (8-bit factors), losses %.1e, gradient %.1e"
          % (tokens, start.elapsed_time(end) * 10, *errors))
    return errors


if __name__ == "__main__":
    main(*[int(a) for a in sys.argv[1:2]])
