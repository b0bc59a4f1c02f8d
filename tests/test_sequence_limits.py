"""The largest calls of the sequence operators: what is one too many for a launch is refused by name, what just fits
gets as far as the device (CPU only)."""

import ctypes

import pytest
import torch

import conv2d_bias_activation_amd as c2d
from test_sequence_abi import _conv, _scan, _w4

FAR = 1 << 50  # stand-in device addresses, far enough apart for rows of any number


def _many(call, **kw):
    """The call on operands that lie far apart."""
    names = {"conv": "x w y", "scan": "u dt a b c y gate", "w4": "x packed y"}[call.__name__.strip("_")].split()
    return call(**{**{n: (i + 1) * FAR for i, n in enumerate(names)}, **kw})


def _conv_rows(n, step):
    d = 2048  # one workgroup of 256 threads for each sequence of one token
    return _many(_conv, step=step, nseq=n, tokens=1, channels=d, state=0, x_batch=d, y_batch=d, x_token=d, y_token=d)


def _scan_rows(n, channels, states, step, packed):
    kw = {f"{t}_{k}": channels for t in ("u", "dt", "gate", "y") for k in ("batch", "token")}
    kw.update({f"{t}_{k}": states for t in "bc" for k in ("batch", "token")})
    if packed:
        kw["offsets"] = 12 * FAR
    return _many(_scan, step=step, nseq=n, tokens=n if packed else 1, channels=channels, states=states, state=0, **kw)


LAUNCHES = [  # rows of a call, the first number too large, the largest that fits
    (lambda n: _conv_rows(n, False), 1 << 24, (1 << 24) - 1),
    (lambda n: _conv_rows(n, True), 1 << 24, (1 << 24) - 1),
    (lambda n: _scan_rows(n, 64, 16, False, False), 1 << 24, (1 << 24) - 1),  # 256 threads each
    (lambda n: _scan_rows(n, 4096, 64, False, True), 1 << 16, (1 << 16) - 1),  # 64 blocks of 1024
    (lambda n: _scan_rows(n, 4096, 256, True, False), 1 << 15, (1 << 15) - 2),  # 1024 of 256 for two
    (lambda n: _many(_w4, rows=n, in_features=256, out_features=32768, x_row=256, y_row=32768), 1 << 18, (1 << 18) - 32),
]


@pytest.mark.parametrize("i", range(len(LAUNCHES)))
def test_one_too_many_for_a_launch_is_unsupported(i):
    call, n, _ = LAUNCHES[i]
    assert call(n) == c2d.EUNSUPPORTED
    assert "too many for one launch" in c2d.last_error()


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="needs a machine without a GPU")
@pytest.mark.parametrize("i", range(len(LAUNCHES)))
def test_what_just_fits_a_launch_reaches_the_device(i):
    call, _, n = LAUNCHES[i]
    assert call(n) == c2d.EHIP, c2d.last_error()


def test_too_many_tokens_are_unsupported():
    more = (1 << 30) + 1
    for call in (lambda: _many(_conv, nseq=more, tokens=1), lambda: _many(_conv, nseq=2, tokens=1 << 30),
                 lambda: _many(_conv, step=True, nseq=more), lambda: _many(_scan, nseq=1, tokens=more),
                 lambda: _many(_scan, step=True, nseq=more), lambda: _many(_w4, rows=more)):
        assert call() == c2d.EUNSUPPORTED
        assert "more than 2^30 tokens" in c2d.last_error()


@pytest.mark.parametrize("n", [(1 << 30) + 1, (1 << 31) - 128, (1 << 31) - 1])
def test_too_wide_is_unsupported(n):
    """Sizes that 32-bit sums with a tile would overflow."""
    size = ctypes.c_size_t(0)
    lib = c2d._load()
    for call in (lambda: _many(_conv, channels=n), lambda: _many(_conv, step=True, channels=n), lambda: _many(_scan, channels=n),
                 lambda: _many(_scan, step=True, channels=n), lambda: _many(_w4, in_features=n, out_features=16),
                 lambda: _many(_w4, in_features=32, out_features=n),
                 lambda: lib.matvec_w4_packed_bytes(16, n, 128, 0, ctypes.byref(size)),
                 lambda: lib.matvec_w4_packed_bytes(n, 16, 128, 0, ctypes.byref(size)),
                 lambda: lib.matvec_w4_pack(FAR, 2 * FAR, None, 3 * FAR, n, 16, 128, c2d.DTYPE_BF16, None)):
        assert call() == c2d.EUNSUPPORTED
        assert "more than 2^30 channels, inputs or outputs" in c2d.last_error()


def test_packed_size_of_the_widest_weights():
    size = ctypes.c_size_t(0)
    packed = c2d._load().matvec_w4_packed_bytes
    assert packed(16, 1 << 30, 128, 0, ctypes.byref(size)) == c2d.OK and size.value == (1 << 23) * (1024 + 32)
    assert packed(1 << 30, 127, 128, 1, ctypes.byref(size)) == c2d.OK and size.value == (1 << 26) * (1024 + 48)
    assert packed((1 << 30) - 1, 1 << 10, 32, 0, ctypes.byref(size)) == c2d.OK and size.value == (1 << 29) * (1024 + 128)
    assert packed((1 << 30) - 1, (1 << 10) + 1, 32, 0, ctypes.byref(size)) == c2d.EUNSUPPORTED
