"""An expert layer with a shared linear, trained and served in 8-bit floats.

The router chooses `top` of `experts` for each token; the order of the rows, the
copies into it and the sums out of it are one launch each, forward and backward.
The shared linear trains in 8 bits: its operands are quantised along whichever
direction a product contracts.  The experts train in 16 bits and are served from
8-bit weights with a scale for each 128 x 128.

    python examples/fp8_experts.py            # on an MI355X
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import structured_sparse_gemm_amd as ssg
from examples.expert_layer import GroupedLinear

once = torch.autograd.function.once_differentiable


class Route(torch.autograd.Function):
    """route; its experts have no gradient.  Gradients of gradients are an error."""

    @staticmethod
    def forward(ctx, logits, k, score, bias, groups, top_groups):
        weights, experts = ssg.route(logits, k, score=score, bias=bias, groups=groups, top_groups=top_groups)
        ctx.save_for_backward(logits, experts)
        ctx.score = score
        ctx.mark_non_differentiable(experts)
        return weights, experts

    @staticmethod
    @once
    def backward(ctx, dweights, _):
        logits, experts = ctx.saved_tensors
        dl = ssg.route_backward(dweights.contiguous(), logits, experts, score=ctx.score)
        return dl, None, None, None, None, None


class Gather(torch.autograd.Function):
    """expert_gather; its gradient is the combine without weights."""

    @staticmethod
    def forward(ctx, x, pos, rows):
        ctx.save_for_backward(pos)
        return ssg.expert_gather(x, pos, rows)

    @staticmethod
    @once
    def backward(ctx, dy):
        return ssg.expert_combine(dy.contiguous(), ctx.saved_tensors[0]), None, None


class Combine(torch.autograd.Function):
    """expert_combine with the gradients of the rows and of the weights."""

    @staticmethod
    def forward(ctx, y, pos, rows, weights):
        ctx.save_for_backward(y, pos, rows, weights)
        return ssg.expert_combine(y, pos, weights)

    @staticmethod
    @once
    def backward(ctx, do):
        y, pos, rows, weights = ctx.saved_tensors
        dy, dw = ssg.expert_combine_backward(do.contiguous(), y, pos, rows, weights)
        return dy, None, None, dw


class Fp8Linear(torch.autograd.Function):
    """x w^T with both rounded to 8 bits; dx and dw are products of the operands
    quantised along the other direction, dw summed in fp32."""

    @staticmethod
    def forward(ctx, x, w):
        ctx.save_for_backward(x, w)
        return ssg.mm_fp8(x, *ssg.fp8_quantize(w, block=128), out_dtype=x.dtype)

    @staticmethod
    @once
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        dy, dx, dw = dy.contiguous(), None, None
        if ctx.needs_input_grad[0]:
            dx = ssg.mm_fp8(dy, *ssg.fp8_quantize(w, block=128, transpose=True), out_dtype=x.dtype)
        if ctx.needs_input_grad[1]:
            e, s = ssg.fp8_quantize(dy, transpose=True)
            dw = ssg.mm_fp8(e, *ssg.fp8_quantize(x, transpose=True), xscales=s).to(w.dtype)
        return dx, dw


class Layer:
    def __init__(self, experts, width, hidden, top=2, score="softmax", groups=1, top_groups=1, dtype=torch.bfloat16,
                 device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weights(*shape):
            w = torch.randn(*shape, generator=gen, device=device) * shape[-1] ** -0.5
            return w.to(dtype).requires_grad_()

        self.experts, self.how = experts, (top, score, torch.zeros(experts, device=device), groups, top_groups)
        self.router, self.shared = weights(experts, width), weights(width, width)
        self.up, self.down = weights(experts, hidden, width), weights(experts, width, hidden)

    def parameters(self):
        return [self.router, self.shared, self.up, self.down]

    def train_forward(self, x):
        weights, experts = Route.apply((x @ self.router.t()).float(), *self.how)
        offs, rows, pos = ssg.expert_order(experts, self.experts)
        h = torch.nn.functional.silu(GroupedLinear.apply(Gather.apply(x, pos, rows), self.up, offs))
        return Combine.apply(GroupedLinear.apply(h, self.down, offs), pos, rows, weights) + Fp8Linear.apply(x, self.shared)

    @torch.no_grad()
    def quantise(self):
        """8-bit copies of the weights, for serve()."""
        self.up8, self.down8, self.shared8 = (ssg.fp8_quantize(w, block=128) for w in (self.up, self.down, self.shared))

    @torch.no_grad()
    def serve(self, x):
        """The layer of one token or of many; nothing waits for the host."""
        top, score, bias, groups, top_groups = self.how
        weights, experts = ssg.route((x @ self.router.t()).float(), top, score=score, bias=bias, groups=groups,
                                     top_groups=top_groups)
        offs, rows, pos = ssg.expert_order(experts, self.experts)
        h = ssg.grouped_mm_fp8(ssg.expert_gather(x, pos, rows), *self.up8, offs, out_dtype=x.dtype)
        y = ssg.grouped_mm_fp8(torch.nn.functional.silu(h), *self.down8, offs, out_dtype=x.dtype)
        return ssg.expert_combine(y, pos, weights) + ssg.mm_fp8(x, *self.shared8, out_dtype=x.dtype)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--experts", type=int, default=32)
    p.add_argument("--width", type=int, default=1024)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args(argv)
    layer = Layer(a.experts, a.width, a.hidden, top=4, score="sigmoid", groups=8 if a.experts % 8 == 0 else 1,
                  top_groups=4 if a.experts % 8 == 0 else 1)
    opt = torch.optim.AdamW(layer.parameters(), lr=1e-3)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.width, generator=gen, device="cuda").bfloat16()
    want = torch.roll(x, 1, dims=1) * 0.5
    loss = None
    for step in range(a.steps):
        loss = (layer.train_forward(x) - want).float().square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        if step % 5 == 0:
            print("step %d: loss %.4f" % (step, loss.item()))
    layer.quantise()
    y = layer.serve(x[:16])
    off = (y - layer.train_forward(x[:16])).float().norm() / y.float().norm()
    print("served from 8-bit weights: %.4f of the norm off" % off.item())
    return loss.item() if loss is not None else None


if __name__ == "__main__":
    main()
