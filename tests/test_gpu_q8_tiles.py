"""Products in 8-bit integers on both sides of the borders between their kernels, against 64 bits."""
import pytest
import torch

import sequence_reference as ref
import test_gpu_q8 as q8

pytestmark = pytest.mark.gpu

c2d = pytest.importorskip("conv2d_bias_activation_amd")


def _check(kind, rows, k, n, act="none", before=False, shift=0):
    dtype = q8.TYPES[kind]
    x = q8._normal(rows + n, rows, k, dtype=dtype)
    wcodes, wscales = q8._weights(n, n, k)
    kw = {"bias": q8._normal(1, n, scale=0.1), "residual": q8._normal(2, rows, n, dtype=dtype),
          "alpha": torch.rand(n, generator=torch.Generator().manual_seed(3)) if act == "prelu" else None}
    want, bound = q8.product(*q8.quantized(x), wcodes, wscales, dtype, act=act, before=before, **kw)
    dev = {name: q8._on(t) for name, t in kw.items()}
    dev["residual"] = q8._wide(kw["residual"], 3, shift)
    out = torch.full((rows + 1, n + 5), 7.0, dtype=dtype, device="cuda")
    y = out[:rows, shift:shift + n]
    c2d.matmul_q8(q8._wide(x, 2, shift), c2d.q8_pack(q8._on(wcodes), q8._on(wscales)), act=act, res_before_act=before, out=y,
                  **dev)
    ref.close(y, want, bound, f"{kind} {rows} x {k} -> {n}")
    assert (out[rows] == 7).all() and (out[:, :shift] == 7).all() and (out[:, shift + n:] == 7).all()


# rows and outputs in 16s: 2 x 256, 2 x 512 and 4 x 256 take the few-rows kernel, the sizes next to them tiles through LDS;
# from 33 to 64 rows, outputs of some 8000 to 11000 are read twice by the one and once by the other
@pytest.mark.parametrize("kind", list(q8.TYPES))
@pytest.mark.parametrize("rows,k,n,more", [
    (37, 100, 10007, {}), (33, 65, 8177, {"act": "prelu"}), (48, 129, 10912, {"act": "relu", "before": True}),
    (33, 64, 8192, {"shift": 1}), (64, 320, 8192, {"act": "silu"}), (49, 200, 8193, {"act": "prelu", "before": True, "shift": 1}),
    (17, 70, 16384, {}), (32, 70, 16385, {"shift": 2}), (65, 130, 5453, {"act": "relu"}), (65, 130, 5441, {}),
    (128, 190, 4096, {"act": "prelu"}), (129, 190, 4096, {"shift": 1}), (127, 90, 4100, {"act": "silu", "before": True})])
def test_next_to_the_few_rows_border(kind, rows, k, n, more):
    _check(kind, rows, k, n, **more)


# one size for each kernel and tile that a product may take, rows, inputs and outputs ending inside it: few rows of 1 x 1, 2 x 1
# and 2 x 2 output tiles, then 64 x 64 (up to 256 workgroups and more), 128 x 128, 128 x 256 and 256 x 256
@pytest.mark.parametrize("kind", list(q8.TYPES))
@pytest.mark.parametrize("rows,k,n", [(9, 70, 2001), (9, 70, 16390), (90, 200, 2030), (199, 65, 4090), (340, 65, 4090),
                                      (1020, 130, 4090), (4090, 70, 2039), (2040, 130, 8190)])
def test_every_tile(kind, rows, k, n):
    _check(kind, rows, k, n, act="prelu", shift=1)


@pytest.mark.parametrize("rows", [3, 40, 340])
def test_rows_without_a_scale_through_the_epilogue(rows):
    """A row with a NaN is NaN before the activation; ReLU makes 0 of a NaN here as in the convolutions, the others keep it."""
    x = q8._normal(1, rows, 70)
    x[1, 5] = float("nan")
    w = c2d.q8_pack(*map(q8._on, q8._weights(1, 4090, 70)))
    r = q8._on(q8._normal(2, rows, 4090))
    alpha = torch.full((4090,), 0.5, device="cuda")
    for act, kw in (("none", {}), ("silu", {}), ("prelu", {"alpha": alpha})):
        y = c2d.matmul_q8(q8._on(x), w, residual=r, act=act, **kw)
        assert torch.isnan(y[1]).all() and not torch.isnan(y[[0, 2]]).any(), act
    y = c2d.matmul_q8(q8._on(x), w, residual=r, act="relu")
    assert torch.equal(y[1], r[1])
    y = c2d.matmul_q8(q8._on(x), w, residual=r, act="relu", res_before_act=True)
    assert (y[1] == 0).all()
