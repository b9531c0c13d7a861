"""The example's functions under gradients that autograd lays out as it likes."""
import pytest
import torch

from examples import fp8_experts as ex
import structured_sparse_gemm_amd as ssg
from tests import _experts as D

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_expanded_and_transposed_gradients(score):
    l = D.randn((20, 12), "f32", 1).cuda()

    def gradients(f, leaf, g):
        leaf = leaf.clone().requires_grad_()
        return torch.autograd.grad(f(leaf), leaf, g)[0]

    route = lambda t: ex.Route.apply(t, 3, score, None, 1, 1)[0]     # noqa: E731
    ones = torch.ones(20, 3).cuda()
    assert torch.equal(gradients(route, l, ones[:1, :1].expand(20, 3)), gradients(route, l, ones))
    g = D.randn((20, 3), "f32", 2).cuda()
    assert torch.equal(gradients(route, l, g.t().contiguous().t()), gradients(route, l, g))

    weights, experts = ssg.route(l, 3, score=score)
    offs, rows, pos = ssg.expert_order(experts, 12)
    x, y = D.randn((20, 40), "f32", 3).cuda(), D.randn((60, 40), "f32", 4).cuda()
    for f, leaf, n in ((lambda t: ex.Gather.apply(t, pos, rows), x, 60), (lambda t: ex.Combine.apply(t, pos, rows, weights), y, 20),
                       (lambda t: ex.Combine.apply(y, pos, rows, t), weights, 20), (lambda t: ex.Fp8Linear.apply(t, y), x, 20)):
        c = f(leaf).shape[1]
        ones, g = torch.ones(n, c).cuda(), D.randn((n, c), "f32", 5).cuda()
        assert torch.equal(gradients(f, leaf, ones[:1, :1].expand(n, c)), gradients(f, leaf, ones))
        assert torch.equal(gradients(f, leaf, g.t().contiguous().t()), gradients(f, leaf, g))
