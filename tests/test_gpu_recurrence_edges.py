"""Calls at the edges of what the recurrence's documentation allows, on the GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu

c2d = pytest.importorskip("conv2d_bias_activation_amd")
DEV = "cuda"


def test_rows_without_a_sequence():
    """Offsets of no sequence: the rows stay as they are and the bias gradient is zero."""
    g = torch.Generator(device=DEV).manual_seed(1)
    x, z, e = (torch.randn(200, 70, generator=g, device=DEV) for _ in range(3))
    offsets = torch.zeros(1, dtype=torch.int32, device=DEV)
    outs = [torch.full_like(x, 7.0) for _ in range(3)]
    c2d.gated_recurrence(x, z, seq_offsets=offsets, out=outs[2])
    got = c2d.gated_recurrence_backward(e, x, z, forget_bias=torch.ones(70, device=DEV), seq_offsets=offsets,
                                        out=(outs[0], outs[1], None))
    assert all((t == 7).all() for t in outs)
    assert got[2] is None and (got[3] == 0).all()


@pytest.mark.parametrize("order", ["batch, which, token", "token, which, batch", "token, batch, which"])
def test_gradients_between_each_other(order):
    """Gradients as interleaved parts of one tensor are those of separate ones."""
    b, t, d = 3, 130, 70
    g = torch.Generator(device=DEV).manual_seed(2)
    x, z, gate, e = (torch.randn(b, t, d, generator=g, device=DEV).bfloat16() for _ in range(4))
    want = c2d.gated_recurrence_backward(e, x, z, gate=gate)
    names = order.split(", ")
    whole = torch.full([{"batch": b, "which": 3, "token": t}[n] for n in names] + [d], float("nan"), dtype=x.dtype, device=DEV)
    parts = whole.permute(names.index("which"), names.index("batch"), names.index("token"), 3).unbind(0)
    got = c2d.gated_recurrence_backward(e, x, z, gate=gate, out=parts)
    for a, w in zip(got[:3], want):
        assert torch.equal(a, w)
