"""The C ABI of rows and products in 8 bits without a GPU: struct layouts and refusals before any launch (CPU only)."""
import ctypes

import pytest
import torch

import conv2d_bias_activation_amd as c2d
from conv2d_bias_activation_amd import sequence
from test_recurrence_abi import _layout_error, _pack

G = 1 << 32  # stand-in device addresses, 4 GiB apart: never dereferenced by these calls
BF16 = c2d.DTYPE_BF16

ROWS = "x packed x_row rows in_features dtype".split()
Q8 = ("x x_packed weights bias alpha residual y x_row residual_row y_row rows in_features out_features act dtype").split()


def test_struct_layouts_match_the_header(tmp_path):
    assert _layout_error(tmp_path, "quantize_rows_args", sequence._QUANTIZE, ROWS) == 0
    assert _layout_error(tmp_path, "matmul_q8_args", sequence._Q8, Q8) == 0


def _rows(**kw):
    v = dict(x=G, packed=2 * G, x_row=256, rows=4, in_features=256, dtype=BF16)
    v.update(kw)
    return c2d._load().quantize_rows(_pack(sequence._QUANTIZE, ROWS, v), None)


def _matmul(size=False, **kw):
    v = dict(x=G, weights=2 * G, y=3 * G, x_row=256, y_row=512, rows=4, in_features=256, out_features=512, dtype=BF16)
    v.update(kw)
    args = _pack(sequence._Q8, Q8, v)
    if size:
        n = ctypes.c_size_t(0)
        rc = c2d._load().matmul_q8_workspace_size(args, ctypes.byref(n))
        return rc if rc else n.value
    return c2d._load().matmul_q8(args, None)


BAD_ROWS = [dict(x=0), dict(packed=0), dict(packed=2 * G + 8), dict(rows=-1), dict(in_features=0), dict(dtype=5), dict(x=G + 1),
            dict(x_row=-1), dict(packed=G), dict(x_row=1 << 50), dict(packed=G + 512)]
BAD_MATMUL = [dict(x=0), dict(x_packed=4 * G), dict(x=0, x_packed=4 * G + 8), dict(weights=0), dict(weights=2 * G + 8), dict(y=0),
              dict(rows=-1), dict(in_features=0), dict(out_features=0), dict(out_features=-3), dict(dtype=9), dict(act=12),
              dict(act=c2d.ACT_PRELU), dict(act=c2d.WEIGHTS_OHWI), dict(x=G + 1), dict(bias=5 * G + 2), dict(alpha=5 * G + 1),
              dict(y_row=511), dict(x_row=-1), dict(y=G), dict(y=2 * G), dict(residual=3 * G, residual_row=512),
              dict(residual=5 * G + 1), dict(bias=3 * G), dict(alpha=3 * G, act=c2d.ACT_PRELU), dict(x=0, x_packed=3 * G)]


@pytest.mark.parametrize("call,kw", [(_rows, k) for k in BAD_ROWS] + [(_matmul, k) for k in BAD_MATMUL])
def test_refused_before_launch(call, kw):
    assert call(**kw) == c2d.EINVAL
    assert c2d.last_error() != ""


@pytest.mark.parametrize("call,kw", [(_rows, dict(in_features=1 << 17)), (_rows, dict(rows=(1 << 30) + 1)),
                                     (_rows, dict(rows=1 << 30, in_features=1 << 11)), (_matmul, dict(in_features=1 << 17)),
                                     (_matmul, dict(out_features=1 << 30, in_features=1 << 11)), (_matmul, dict(rows=1 << 30, in_features=1 << 11))])
def test_too_large_is_unsupported(call, kw):
    assert call(**kw) == c2d.EUNSUPPORTED


def test_too_many_threads_are_refused():
    assert _rows(rows=1 << 27, in_features=64, x_row=64, packed=100 * G) == c2d.EUNSUPPORTED and "2^32" in c2d.last_error()
    many = dict(x=0, x_packed=1 << 45, rows=1 << 20, out_features=1 << 20, in_features=64, y=1 << 50, y_row=1 << 20)
    assert _matmul(**many) == c2d.EUNSUPPORTED and "2^32" in c2d.last_error()


def test_sizes():
    n = ctypes.c_size_t(0)
    size = c2d._load().q8_packed_bytes
    assert size(16, 64, ctypes.byref(n)) == c2d.OK and n.value == 1024 + 64
    assert size(17, 65, ctypes.byref(n)) == c2d.OK and n.value == 4 * 1024 + 128
    assert size(0, 65, ctypes.byref(n)) == c2d.OK and n.value == 0
    assert size(17, 1 << 17, ctypes.byref(n)) == c2d.EUNSUPPORTED
    assert size(17, 0, ctypes.byref(n)) == c2d.EINVAL and size(17, 1, None) == c2d.EINVAL
    assert _matmul(size=True, rows=17) >= 2 * 4 * 1024 + 128
    assert _matmul(size=True, rows=4) == 0 and _matmul(size=True, rows=4, in_features=8193, x_row=8193) > 0
    assert _matmul(size=True, x=0, x_packed=4 * G) == 0 and _matmul(size=True, rows=0) == 0


def test_pack_refusals():
    pack, unpack = c2d._load().q8_pack, c2d._load().q8_unpack
    assert pack(G, 2 * G, 3 * G + 8, 16, 64, None) == c2d.EINVAL
    assert pack(G, 2 * G + 2, 3 * G, 16, 64, None) == c2d.EINVAL
    assert pack(None, 2 * G, 3 * G, 16, 64, None) == c2d.EINVAL
    assert pack(G, 2 * G, G, 16, 64, None) == c2d.EINVAL
    assert pack(G, 2 * G, 3 * G, -1, 64, None) == c2d.EINVAL
    assert pack(G, 2 * G, 3 * G, 1, 1 << 17, None) == c2d.EUNSUPPORTED
    assert unpack(G, 2 * G, None, 16, 64, None) == c2d.EINVAL
    assert unpack(G + 8, 2 * G, 3 * G, 16, 64, None) == c2d.EINVAL
    assert unpack(G, G + 512, 3 * G, 16, 64, None) == c2d.EINVAL
    assert unpack(G, 2 * G, 2 * G + 64, 16, 64, None) == c2d.EINVAL
    assert pack(None, None, None, 0, 64, None) == c2d.OK and unpack(None, None, None, 0, 64, None) == c2d.OK


def test_too_small_a_workspace_is_refused_by_name():
    c2d._load().conv2d_set_workspace(None, 0)
    assert _matmul(rows=40) == c2d.EUNSUPPORTED
    assert "needs a workspace" in c2d.last_error()


def test_nothing_to_do_is_fine_without_a_device():
    assert _rows(rows=0, x=0, packed=0) == c2d.OK
    assert _matmul(rows=0, x=0, y=0) == c2d.OK


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="needs a machine without a GPU")
def test_no_device_returns_ehip_not_a_crash():
    for call in (_rows, _matmul, lambda: _matmul(x=0, x_packed=4 * G), lambda: _matmul(x=0, x_packed=4 * G, rows=2000, y_row=600),
                 lambda: c2d._load().q8_pack(G, 2 * G, 3 * G, 16, 64, None),
                 lambda: c2d._load().q8_unpack(G, 2 * G, 3 * G, 16, 64, None)):
        assert call() == c2d.EHIP
        assert c2d.last_error() != ""


def test_binding_refuses():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="expected a GPU"):
        c2d.quantize_rows(x)
    with pytest.raises(ValueError, match="expected a GPU"):
        c2d.q8_pack(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(ValueError, match="unsupported dtype"):
        c2d.quantize_rows(x.double())
    with pytest.raises(ValueError, match="unsupported dtype"):
        c2d.q8_pack(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4), dtype=torch.float64)
