"""The example's differentiable recurrence outside a plain training step."""
import pytest
import torch

from test_gpu_gated_recurrence_example import module  # noqa: F401

pytestmark = pytest.mark.gpu


def test_second_derivatives_are_refused(module):  # noqa: F811
    """The gradient has no history; a loss that contains it would otherwise lose that part in silence."""
    x, z, gate = (torch.randn(1, 20, 8, device="cuda", requires_grad=True) for _ in range(3))
    y = module.recurrence(x, z, gate, torch.zeros(8, device="cuda"))
    (gx,) = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (gx.square().sum() + x.square().sum()).backward()


def test_inputs_that_need_no_gradient(module):  # noqa: F811
    torch.manual_seed(1)
    x, z, gate = (torch.randn(2, 30, 8, device="cuda") for _ in range(3))
    bias = torch.rand(8, device="cuda")
    leaves = [t.clone().requires_grad_() for t in (x, z, gate, bias)]
    module.recurrence(*leaves).square().sum().backward()
    only = z.clone().requires_grad_()
    module.recurrence(x, only, gate, bias).square().sum().backward()
    assert torch.equal(only.grad, leaves[1].grad)
