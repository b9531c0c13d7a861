"""The example's expert layer against the formulas in 64 bits."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
ex = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ex)


def test_route_cpu():
    torch.manual_seed(0)
    logits = torch.randn(37, 5)
    logits[:, 3] = -100.0                                  # an expert without tokens
    token, weight, offs = ex.route(logits, 2)
    assert offs.dtype == torch.int32 and offs[0] == 0 and offs[-1] == 74 and offs[3] == offs[4]
    chosen = logits.topk(2, dim=1).indices
    for e in range(5):
        rows = token[offs[e]:offs[e + 1]]
        assert sorted(rows.tolist()) == sorted((chosen == e).any(dim=1).nonzero().flatten().tolist())
    total = torch.zeros(37).index_add(0, token, weight)
    assert torch.allclose(total, torch.ones(37))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,M,K,sizes", [(1, 40, 24, [0, 1]), (70, 129, 66, [33, 0, 37]), (9, 8, 8, [0, 0, 0])])
def test_gradients_of_the_linear(rows, M, K, sizes):
    """Outputs and gradients, and the gradients against differences of the
    64-bit formula.  fp16 operands; each 16-bit result is half a step off, and
    the sums of n exact products n + 16 steps of 2^-23 of their magnitudes."""
    torch.manual_seed(rows)
    offs = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32)
    x = torch.randn(rows, K).half().cuda().requires_grad_()
    w = torch.randn(len(sizes), M, K).half().cuda().requires_grad_()
    g = torch.randn(rows, M).half().cuda()
    y = ex.GroupedLinear.apply(x, w, offs.cuda())
    y.backward(g)
    x64, w64, g64 = x.detach().cpu().double(), w.detach().cpu().double(), g.cpu().double()
    eps = torch.finfo(torch.float16).eps

    def near(got, ref, mag, n):
        tol = (n + 16) * 2.0 ** -23 * mag
        tol = tol + (ref.abs() + tol) * eps / 2 + torch.finfo(torch.float16).smallest_normal * eps / 2
        assert ((got.detach().cpu().double() - ref).abs() <= tol).all()

    def forward(x_, w_):
        out = torch.zeros(rows, M, dtype=torch.float64)
        for e in range(len(sizes)):
            s = slice(offs[e], offs[e + 1])
            out[s] = x_[s] @ w_[e].t()
        return out

    near(y, forward(x64, w64), forward(x64.abs(), w64.abs()), K)
    dx, dxm = torch.zeros_like(x64), torch.zeros_like(x64)
    dw, dwm = torch.zeros_like(w64), torch.zeros_like(w64)
    for e in range(len(sizes)):
        s = slice(offs[e], offs[e + 1])
        dx[s], dxm[s] = g64[s] @ w64[e], g64[s].abs() @ w64[e].abs()
        dw[e], dwm[e] = g64[s].t() @ x64[s], g64[s].abs().t() @ x64[s].abs()
    near(x.grad, dx, dxm, M)
    near(w.grad, dw, dwm, rows)
    # the loss is linear in x and in w: a difference of any length is its slope
    for t, grad, bound in ((x64, x.grad, dxm), (w64, w.grad, dwm)):
        d = torch.randn_like(t)
        a, b = (t + d, w64) if t is x64 else (x64, t + d)
        slope = ((forward(a, b) - forward(x64, w64)) * g64).sum()
        have = (grad.cpu().double() * d).sum()
        n = max(M, rows)
        tol = (d.abs() * ((n + 17) * 2.0 ** -23 * bound + (bound + 1) * eps / 2)).sum() + 1e-9 * d.abs().sum()
        assert (slope - have).abs() <= tol


@pytest.mark.gpu
def test_example_runs():
    losses, errors = ex.main(["--experts", "4", "--width", "256", "--hidden", "384", "--tokens", "300", "--steps", "15"])
    assert losses[-1] < losses[0]
    # an element's rounding is at most a quarter of it or half the smallest step;
    # over a layer of two products the errors stay well below the signal
    assert all(0 < e < 0.5 for e in errors.values())
    assert errors["16-bit activations"] < errors["mx4 activations"]
