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
