"""The binding on a torch without the private names that its short paths use."""
import os
import subprocess
import sys

import pytest
import torch

import conv2d_bias_activation_amd as c2d
from conv2d_bias_activation_amd import sequence

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_imports_and_plans():
    """The host-only calls of the package need none of them."""
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import conv2d_bias_activation_amd as c2d\n"
            "print(c2d.plan(1, 8, 8, 64, 64, 3, 3, 1, 1, c2d.ACT_RELU, c2d.LAYOUT_NHWC, c2d.DTYPE_BF16))\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=200)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip()


@pytest.mark.gpu
def test_calls_take_the_public_way(monkeypatch):
    monkeypatch.setattr(sequence, "_raw_stream", sequence._stream_handle)
    monkeypatch.setattr(sequence, "_current_device", torch.cuda.current_device)
    side = torch.cuda.Stream()
    x, w = torch.ones(1, 700, 64, device="cuda"), torch.ones(64, 4, device="cuda")
    A, b = -torch.ones(64, 16, device="cuda"), torch.ones(1, 700, 1, 16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        y = c2d.causal_conv1d(x, w)
        z = c2d.selective_scan(x, x, A, b, b)
    side.synchronize()
    assert (y[0, 3:] == 4).all() and torch.isfinite(z).all()
    assert (torch.cuda.current_device(), side.cuda_stream) in c2d._ws_cache
