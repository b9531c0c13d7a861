"""An expert layer trained with 16-bit weights and served with mx4 weights.

Each token goes to `top` of `experts` two-layer networks.  The tokens are
sorted by expert once a layer; the grouped products then take all experts in
one launch, whatever the router chose, without the host learning the sizes.

    python examples/expert_layer.py            # on an MI355X
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import structured_sparse_gemm_amd as ssg


class GroupedLinear(torch.autograd.Function):
    """grouped_mm with its gradients; weight gradients come in fp32 and are
    rounded to the weights' type.  The gradients have no gradients of their own:
    asking for them is an error."""

    @staticmethod
    def forward(ctx, x, w, offs):
        ctx.save_for_backward(x, w, offs)
        return ssg.grouped_mm(x, w, offs)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w, offs = ctx.saved_tensors
        dy = dy.contiguous()
        dx = ssg.grouped_mm_dx(dy, w, offs) if ctx.needs_input_grad[0] else None
        dw = None
        if ctx.needs_input_grad[1]:
            dw = ssg.grouped_mm_dw(dy, x, offs, out_dtype=torch.float32).to(w.dtype)
        return dx, dw, None


def route(logits, top):
    """(token of each sorted row, its weight, offsets [E + 1] on the device)."""
    weight, expert = torch.softmax(logits.float(), dim=1).topk(top, dim=1)
    weight = weight / weight.sum(dim=1, keepdim=True)
    order = torch.argsort(expert.flatten(), stable=True)
    bounds = torch.arange(logits.shape[1] + 1, device=logits.device)
    offs = torch.searchsorted(expert.flatten()[order].contiguous(), bounds).to(torch.int32)
    return order // top, weight.flatten()[order], offs


def combine(rows, token, weight, tokens):
    """Sum of each token's expert outputs."""
    out = torch.zeros(tokens, rows.shape[1], dtype=torch.float32, device=rows.device)
    return out.index_add(0, token, rows.float() * weight[:, None])


class ExpertLayer:
    def __init__(self, experts, width, hidden, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weights(*shape):
            w = torch.randn(*shape, generator=gen, device=device) * shape[-1] ** -0.5
            return w.to(dtype).requires_grad_()

        self.router = weights(experts, width)
        self.up, self.down = weights(experts, hidden, width), weights(experts, width, hidden)

    def parameters(self):
        return [self.router, self.up, self.down]

    def train_forward(self, x, top=2):
        token, weight, offs = route(x @ self.router.t(), top)
        h = GroupedLinear.apply(x[token], self.up, offs)
        y = GroupedLinear.apply(torch.nn.functional.silu(h), self.down, offs)
        return combine(y, token, weight, x.shape[0])

    def quantise(self):
        """mx4 copies of the expert weights, for serve()."""
        with torch.no_grad():
            self.up4, self.down4 = ssg.mx4_quantize(self.up), ssg.mx4_quantize(self.down)
        return self

    @torch.no_grad()
    def serve(self, x, top=2, quantise_activations=False):
        """With mx4 weights; the activations 16-bit (decode), or mx4 too (prefill)."""
        token, weight, offs = route(x @ self.router.t(), top)

        def product(a, w4):
            if quantise_activations:
                a4, scales = ssg.mx4_quantize(a)
                return ssg.grouped_mm_mx4(a4, *w4, offs, xscales=scales, out_dtype=x.dtype)
            return ssg.grouped_mm_mx4(a, *w4, offs, out_dtype=x.dtype)

        h = torch.nn.functional.silu(product(x[token], self.up4))
        return combine(product(h, self.down4), token, weight, x.shape[0])


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=40)
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.width, generator=gen, device="cuda").to(torch.bfloat16)
    goal = torch.tanh(x.float() @ torch.randn(a.width, a.width, generator=gen, device="cuda") * a.width ** -0.5)
    layer = ExpertLayer(a.experts, a.width, a.hidden)
    opt = torch.optim.AdamW(layer.parameters(), lr=1e-3, foreach=True)
    losses = []
    for _ in range(a.steps):
        loss = (layer.train_forward(x) - goal).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    with torch.no_grad():
        full = layer.train_forward(x)
    layer.quantise()
    errors = {}
    for name, quantised in (("16-bit activations", False), ("mx4 activations", True)):
        y = layer.serve(x, quantise_activations=quantised)
        errors[name] = float((y - full).norm() / full.norm())
    one = layer.serve(x[:1])                               # a single token
    print("loss %.4f -> %.4f; mx4 weights against 16-bit ones: %s; one token %s"
          % (losses[0], losses[-1], ", ".join("%.3f with %s" % (e, n) for n, e in errors.items()), tuple(one.shape)))
    return [float(l) for l in losses], errors


if __name__ == "__main__":
    main()
