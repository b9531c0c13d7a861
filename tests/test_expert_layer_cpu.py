"""The example's grouped linear layer under autograd, with plain products in the
place of the library's."""
import pytest
import torch

from tests.test_gpu_expert_layer import ex


class Plain:
    @staticmethod
    def grouped_mm(x, w, offs):
        return torch.cat([x[a:b] @ w[e].t() for e, (a, b) in enumerate(zip(offs[:-1], offs[1:]))])

    @staticmethod
    def grouped_mm_dx(dy, w, offs):
        return torch.cat([dy[a:b] @ w[e] for e, (a, b) in enumerate(zip(offs[:-1], offs[1:]))])

    @staticmethod
    def grouped_mm_dw(dy, x, offs, out_dtype):
        return torch.stack([dy[a:b].t() @ x[a:b] for a, b in zip(offs[:-1], offs[1:])])


@pytest.fixture
def layer(monkeypatch):
    monkeypatch.setattr(ex, "ssg", Plain)
    gen = torch.Generator().manual_seed(1)
    x, w = (torch.randn(*n, generator=gen, dtype=torch.float64).requires_grad_() for n in ((7, 5), (3, 4, 5)))
    return x, w, torch.tensor([0, 3, 3, 7])


def test_gradients(layer):
    x, w, offs = layer
    assert torch.autograd.gradcheck(lambda a, b: ex.GroupedLinear.apply(a, b, offs), (x, w))


def test_second_gradients_are_an_error(layer):
    # through a loss that is not linear in the layer's output, where they exist
    x, w, offs = layer
    dx, = torch.autograd.grad(ex.GroupedLinear.apply(x, w, offs).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.sum().backward()
