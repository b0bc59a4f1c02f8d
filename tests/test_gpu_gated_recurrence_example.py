"""The example block: a prompt and then single tokens give what one long prompt gives, and its training step's gradients
are those of the definition."""
import importlib.util
import os

import pytest
import torch

import recurrence_reference as rec
import sequence_reference as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def module():
    path = os.path.join(ROOT, "examples", "gated_recurrence_block.py")
    spec = importlib.util.spec_from_file_location("gated_recurrence_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_tokens_continue_a_prompt(module):
    """Up to the recurrence both paths have the same bits (rows are quantized alone, sums are exact); its outputs may then
    differ by a rounding to bf16 and so a code by one, which moves a row of codes by at most its scale, a 127th of its
    largest value, say six times its root mean square: 6 / 127 of the projection's part of the output at worst, and two
    roundings. The recurrence's own states differ by 32-bit roundings, twelve a token over some 400 tokens."""
    worst, drift, grads = module.main(["--model", "256", "--prompt", "150", "--tokens", "12", "--batch", "3"])
    assert worst < 6 / 127 + 2 * 2.0 ** -8
    assert drift[0] == 0
    assert drift[1] < 12 * 400 * 2.0 ** -24
    assert set(grads) == {"into.weight", "out.weight", "forget_bias"}
    for name, g in grads.items():
        assert torch.isfinite(g).all() and g.abs().max() > 0, name


def test_gradients_of_the_differentiable_recurrence(module):
    g = torch.Generator().manual_seed(3)
    n, t, d = 2, 70, 24
    x, z, gate, e = (torch.randn(n, t, d, generator=g) for _ in range(4))
    bias = torch.rand(d, generator=g) * 6
    leaves = [v.cuda().requires_grad_() for v in (x, z, gate, bias)]
    y = module.recurrence(*leaves)
    y.backward(e.cuda())
    flat = [v.reshape(n * t, d) for v in (e, x, z, gate)]
    want = rec.backward(*flat, bias, True, None, None, None, [t] * n)
    for name, leaf, (value, bound) in zip(["x", "forget", "gate", "bias"], leaves, want):
        ref.close(leaf.grad.reshape(value.shape), value, bound, name)


def test_a_projection_feeds_it_slices(module):
    """Values, gates and their gradients as thirds of one projection, against 64-bit differentiation of the whole block."""
    torch.manual_seed(5)
    block = module.TrainedBlock(32, 16).cuda()
    x = torch.randn(2, 65, 32, device="cuda")
    block(x).square().sum().backward()
    p = {k: v.detach().cpu().double().requires_grad_() for k, v in block.named_parameters()}
    xd = x.cpu().double()
    value, forget, gate = (xd @ p["into.weight"].t()).chunk(3, -1)
    f = torch.sigmoid(forget + p["forget_bias"])
    h, ys = torch.zeros(2, 16, dtype=torch.float64), []
    for i in range(65):
        h = f[:, i] * h + (1 - f[:, i]) * value[:, i]
        ys.append(h)
    y = torch.stack(ys, 1) * gate * torch.sigmoid(gate)
    (xd + y @ p["out.weight"].t()).square().sum().backward()
    for name, q in block.named_parameters():
        want = p[name].grad
        # sums of some thousand products of 32-bit values with 32-bit errors of some ten roundings each
        assert (q.grad.cpu().double() - want).abs().max() <= 4000 * ref.U32 * want.abs().max(), name
