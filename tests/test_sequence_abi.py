"""The sequence operators' C ABI without a GPU: exports, struct layouts, and what the entry points refuse before
anything is launched (CPU only)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import conv2d_bias_activation_amd as c2d
from conv2d_bias_activation_amd import sequence

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sequence_ops.h")
G = 1 << 32  # stand-in device addresses, 4 GiB apart: never dereferenced by these calls
BF16, F16, F32 = c2d.DTYPE_BF16, c2d.DTYPE_F16, c2d.DTYPE_F32

CONV = ("x w bias alpha state y offsets slots x_batch x_token y_batch y_token tokens nseq state_rows channels width act "
        "dtype fresh").split()
SCAN = ("u dt a b c skip gate dt_bias state y offsets slots u_batch u_token dt_batch dt_token b_batch b_token c_batch "
        "c_token gate_batch gate_token y_batch y_token tokens longest nseq state_rows channels groups states softplus dtype "
        "fresh").split()
W4 = ("x packed bias alpha residual y x_row residual_row y_row rows in_features out_features group has_zeros act "
      "dtype").split()
STRUCTS = {"causal_conv1d_args": (sequence._CONV, CONV), "selective_scan_args": (sequence._SCAN, SCAN),
           "matvec_w4_args": (sequence._W4, W4)}


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^int (\w+)\s*\(", text, flags=re.M))
    assert names == set(c2d.SEQUENCE_SIGNATURES)
    lib = ctypes.CDLL(c2d.library_path())
    for name in names:
        assert hasattr(lib, name), name


def test_struct_layouts_match_the_header(tmp_path):
    """A struct packed by the binding with 1, 2, 3, ... reads back so, field by field, in C."""
    checks = []
    for name, (layout, fields) in STRUCTS.items():
        blob = layout.pack(*range(1, len(fields) + 1))
        body = ",".join(str(b) for b in blob)
        checks.append(f"  {{ static const _Alignas(16) unsigned char p[] = {{{body}}};\n"
                      f"    const {name} *a = (const {name} *)p; if (sizeof p != sizeof *a) return 1;\n" +
                      "".join(f"    if ((long long)a->{f} != {i + 1}) return {i + 2};\n" for i, f in enumerate(fields)) +
                      "  }\n")
    src = tmp_path / "layout.c"
    src.write_text('#include "sequence_ops.h"\nint main(void) {\n' + "".join(checks) + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def _pack(layout, fields, values):
    assert set(values) <= set(fields), set(values) - set(fields)
    return layout.pack(*(values.get(f, 0) for f in fields))


def _conv(step=False, **kw):
    d = 64
    v = dict(x=G, w=2 * G, y=3 * G, state=4 * G, x_batch=100 * d, x_token=d, y_batch=100 * d, y_token=d, tokens=100, nseq=2,
             state_rows=5, channels=d, width=4, act=c2d.ACT_SILU, dtype=BF16)
    if step:
        v.update(tokens=1)
    v.update(kw)
    fn = c2d._load().causal_conv1d_step if step else c2d._load().causal_conv1d
    return fn(_pack(sequence._CONV, CONV, v), None)


def _scan(step=False, **kw):
    d = 64
    row = dict(batch=100 * d, token=d)
    v = dict(u=G, dt=2 * G, a=3 * G, b=4 * G, c=5 * G, state=6 * G, y=7 * G, gate=8 * G, b_batch=1600, b_token=16,
             c_batch=1600, c_token=16, tokens=100, nseq=2, state_rows=5, channels=d, groups=1, states=16, dtype=BF16)
    v.update({f"{t}_{k}": row[k] for t in ("u", "dt", "gate", "y") for k in row})
    if step:
        v.update(tokens=1)
    v.update(kw)
    fn = c2d._load().selective_scan_step if step else c2d._load().selective_scan
    return fn(_pack(sequence._SCAN, SCAN, v), None)


def _w4(**kw):
    v = dict(x=G, packed=2 * G, y=3 * G, x_row=256, y_row=512, rows=4, in_features=256, out_features=512, group=64, dtype=BF16)
    v.update(kw)
    return c2d._load().matvec_w4(_pack(sequence._W4, W4, v), None)


BAD_CONV = [dict(x=0), dict(w=0), dict(y=0), dict(channels=0), dict(width=1), dict(width=5), dict(nseq=-1), dict(tokens=-1),
            dict(state_rows=-1), dict(dtype=3), dict(act=9), dict(act=c2d.ACT_RELU | c2d.RES_BEFORE_ACT),
            dict(act=c2d.ACT_PRELU), dict(x=G + 1), dict(state=4 * G + 1), dict(offsets=5 * G + 2), dict(bias=5 * G + 1),
            dict(x_token=-64), dict(x_batch=1 << 50), dict(y_token=63), dict(y_batch=64 * 99), dict(y=G + 128),
            dict(state=3 * G + 2), dict(state=G), dict(bias=3 * G), dict(slots=3 * G), dict(offsets=4 * G)]
BAD_SCAN = [dict(u=0), dict(dt=0), dict(a=0), dict(b=0), dict(c=0), dict(y=0), dict(channels=0), dict(groups=0),
            dict(groups=3), dict(states=0), dict(states=257), dict(longest=-1), dict(nseq=-1), dict(tokens=-1), dict(dtype=7),
            dict(u=G + 1), dict(a=3 * G + 2), dict(state=6 * G + 2), dict(b_token=-1), dict(c_batch=1 << 50),
            dict(y_token=32), dict(y=G), dict(y=8 * G + 64), dict(y=3 * G), dict(state=3 * G), dict(state=7 * G),
            dict(skip=7 * G), dict(dt_bias=6 * G), dict(slots=7 * G), dict(offsets=6 * G)]
BAD_W4 = [dict(x=0), dict(packed=0), dict(y=0), dict(packed=2 * G + 8), dict(group=16), dict(group=96), dict(rows=-1),
          dict(in_features=0), dict(out_features=-4), dict(dtype=F32), dict(act=12), dict(act=c2d.ACT_PRELU),
          dict(act=c2d.WEIGHTS_OHWI), dict(x=G + 1), dict(bias=5 * G + 2), dict(y_row=511), dict(x_row=-1), dict(y=G),
          dict(y=2 * G), dict(residual=3 * G, residual_row=512), dict(bias=3 * G)]


@pytest.mark.parametrize("call,kw", [(_conv, k) for k in BAD_CONV] + [(_scan, k) for k in BAD_SCAN] +
                         [(_w4, k) for k in BAD_W4])
def test_refused_before_launch(call, kw):
    assert call(**kw) == c2d.EINVAL
    assert c2d.last_error() != ""


@pytest.mark.parametrize("call,kw", [
    (_conv, dict(tokens=1 << 30, nseq=2, x_batch=0, x_token=0)), (_conv, dict(nseq=(1 << 30) + 1)),
    (_conv, dict(tokens=(1 << 30) - 1, nseq=1, channels=1 << 16, x_token=0, y_token=1 << 14, offsets=9 * G)),
    (_scan, dict(tokens=(1 << 30) + 1, nseq=1)), (_scan, dict(tokens=1, nseq=1 << 29, channels=1 << 20, u_batch=0)),
    (_w4, dict(out_features=1 << 30, in_features=1 << 30)), (_w4, dict(rows=(1 << 30) + 1, x_row=0))])
def test_too_large_is_unsupported(call, kw):
    assert call(**kw) in (c2d.EUNSUPPORTED, c2d.EINVAL)
    assert c2d.last_error() != ""


def test_single_token_calls_take_no_offsets():
    assert _conv(step=True, offsets=9 * G) == c2d.EINVAL
    assert _conv(step=True, tokens=2) == c2d.EINVAL
    assert _scan(step=True, offsets=9 * G) == c2d.EINVAL
    assert "one token" in c2d.last_error()
    assert c2d._load().causal_conv1d(None, None) == c2d.EINVAL


def test_nothing_to_do_is_fine_without_a_device():
    assert _conv(nseq=0, x=0, y=0) == c2d.OK
    assert _scan(nseq=0, u=0, dt=0, b=0, c=0, y=0) == c2d.OK
    assert _w4(rows=0, x=0, y=0) == c2d.OK


def test_packed_size():
    n = ctypes.c_size_t(0)
    size = c2d._load().matvec_w4_packed_bytes
    assert size(16, 128, 128, 0, ctypes.byref(n)) == c2d.OK and n.value == 1024 + 16 * 2
    assert size(17, 129, 32, 1, ctypes.byref(n)) == c2d.OK and n.value == 4 * (1024 + 16 * 4 * 3)
    assert size(17, 129, 48, 1, ctypes.byref(n)) == c2d.EINVAL
    assert size(17, 129, 32, 1, None) == c2d.EINVAL
    pack = c2d._load().matvec_w4_pack
    assert pack(G, 2 * G, None, 3 * G + 8, 16, 128, 64, BF16, None) == c2d.EINVAL
    assert pack(G, 2 * G, None, G, 16, 128, 64, BF16, None) == c2d.EINVAL
    assert pack(G, 2 * G, None, 3 * G, 16, 128, 64, F32, None) == c2d.EINVAL
    assert pack(None, 2 * G, None, 3 * G, 16, 128, 64, BF16, None) == c2d.EINVAL


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="needs a machine without a GPU")
def test_no_device_returns_ehip_not_a_crash():
    calls = [_conv, _scan, _w4, lambda: _conv(step=True), lambda: _scan(step=True), lambda: _conv(offsets=9 * G),
             lambda: _scan(offsets=9 * G, softplus=1, slots=10 * G),
             lambda: c2d._load().matvec_w4_pack(G, 2 * G, None, 3 * G, 16, 128, 64, BF16, None)]
    for call in calls:
        assert call() == c2d.EHIP
        assert c2d.last_error() != ""


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(2, 5, 8)
    with pytest.raises(ValueError, match="expected a GPU"):
        c2d.causal_conv1d(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="unsupported dtype"):
        c2d.selective_scan(x.double(), x, torch.zeros(8, 4), x, x)
    with pytest.raises(ValueError, match="expected bfloat16 or float16"):
        c2d.w4_pack(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1))
