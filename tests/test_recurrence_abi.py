"""The recurrence's C ABI without a GPU: struct layouts, and what the entry points refuse before anything is launched
(CPU only)."""
import ctypes
import os
import subprocess

import pytest
import torch

import conv2d_bias_activation_amd as c2d
from conv2d_bias_activation_amd import sequence

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
G = 1 << 32  # stand-in device addresses, 4 GiB apart: never dereferenced by these calls
D = 64

REC = ("x forget gate forget_bias state y offsets slots x_batch x_token forget_batch forget_token gate_batch gate_token "
       "y_batch y_token tokens longest nseq state_rows channels coupled dtype fresh").split()
BACK = ("grad x forget gate forget_bias state grad_state grad_x grad_forget grad_gate grad_forget_bias offsets slots "
        "grad_batch grad_token x_batch x_token forget_batch forget_token gate_batch gate_token grad_x_batch grad_x_token "
        "grad_forget_batch grad_forget_token grad_gate_batch grad_gate_token tokens longest nseq state_rows channels coupled "
        "dtype").split()


def _layout_error(tmp_path, name, layout, fields):
    """0 if a struct packed by the binding with 1, 2, 3, ... reads back so, field by field, in C."""
    body = ",".join(str(b) for b in layout.pack(*range(1, len(fields) + 1)))
    src = tmp_path / f"{name}.c"
    src.write_text('#include "sequence_ops.h"\nint main(void) {\n'
                   f"  static const _Alignas(16) unsigned char p[] = {{{body}}};\n"
                   f"  const {name} *a = (const {name} *)p;\n  if (sizeof p != sizeof *a) return 1;\n" +
                   "".join(f"  if ((long long)a->{f} != {i + 1}) return {i + 2};\n" for i, f in enumerate(fields)) +
                   "  return 0;\n}\n")
    exe = tmp_path / name
    subprocess.run(["gcc", "-std=c11", "-I", HEADER, str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)]).returncode


def test_struct_layouts_match_the_header(tmp_path):
    assert _layout_error(tmp_path, "gated_recurrence_args", sequence._REC, REC) == 0
    assert _layout_error(tmp_path, "gated_recurrence_backward_args", sequence._REC_BACK, BACK) == 0


def _pack(layout, fields, values):
    assert set(values) <= set(fields), set(values) - set(fields)
    return layout.pack(*(values.get(f, 0) for f in fields))


def _rec(step=False, size=False, **kw):
    v = dict(x=G, forget=2 * G, gate=3 * G, forget_bias=4 * G, state=5 * G, y=6 * G, tokens=100, nseq=2, state_rows=5, channels=D,
             coupled=1, dtype=c2d.DTYPE_BF16)
    v.update({f"{t}_{k}": n for t in ("x", "forget", "gate", "y") for k, n in (("batch", 100 * D), ("token", D))})
    if step:
        v.update(tokens=1)
    v.update(kw)
    args = _pack(sequence._REC, REC, v)
    if size:
        n = ctypes.c_size_t(0)
        rc = c2d._load().gated_recurrence_workspace_size(args, ctypes.byref(n))
        return rc if rc else n.value
    return (c2d._load().gated_recurrence_step if step else c2d._load().gated_recurrence)(args, None)


def _back(size=True, **kw):
    v = dict(grad=G, x=2 * G, forget=3 * G, gate=4 * G, forget_bias=5 * G, state=6 * G, grad_state=7 * G, grad_x=8 * G,
             grad_forget=9 * G, grad_gate=10 * G, grad_forget_bias=11 * G, tokens=100, nseq=2, state_rows=5, channels=D,
             coupled=1, dtype=c2d.DTYPE_BF16)
    rows = ("grad", "x", "forget", "gate", "grad_x", "grad_forget", "grad_gate")
    v.update({f"{t}_{k}": n for t in rows for k, n in (("batch", 100 * D), ("token", D))})
    v.update(kw)
    args = _pack(sequence._REC_BACK, BACK, v)
    if size:
        n = ctypes.c_size_t(0)
        rc = c2d._load().gated_recurrence_backward_workspace_size(args, ctypes.byref(n))
        return rc if rc else n.value
    return c2d._load().gated_recurrence_backward(args, None)


BAD = [dict(channels=0), dict(nseq=-1), dict(tokens=-1), dict(state_rows=-1), dict(longest=-1), dict(dtype=3), dict(x=0),
       dict(forget=0), dict(x=G + 1), dict(gate=4 * G + 1), dict(forget_bias=5 * G + 2), dict(state=6 * G + 2),
       dict(offsets=12 * G + 2), dict(slots=12 * G + 1), dict(x_token=-1), dict(forget_batch=-64), dict(x_batch=1 << 50)]
BAD_REC = BAD + [dict(y=0), dict(y_token=63), dict(y_batch=64 * 99), dict(y=G), dict(y=2 * G + 128), dict(y=3 * G), dict(y=4 * G),
                 dict(y=5 * G), dict(slots=6 * G), dict(state=G), dict(state=4 * G), dict(offsets=5 * G)]
BAD_BACK = BAD + [dict(grad=0), dict(grad_x=0), dict(grad_forget=0), dict(grad_gate=0), dict(gate=0),
                  dict(grad_forget_bias=11 * G + 1), dict(grad_state=7 * G + 2), dict(grad_x_token=63),
                  dict(grad_gate_batch=64 * 99), dict(grad_x=G), dict(grad_forget=4 * G), dict(grad_gate=10 * G + 1),
                  dict(grad_x=9 * G), dict(grad_forget=10 * G + 2 * D * 50), dict(grad_x=6 * G), dict(grad_gate=7 * G),
                  dict(grad_forget_bias=8 * G), dict(grad_forget_bias=5 * G), dict(grad_state=6 * G), dict(grad_state=G),
                  dict(slots=10 * G), dict(offsets=7 * G)]


@pytest.mark.parametrize("call,kw", [(_rec, k) for k in BAD_REC] + [(_back, k) for k in BAD_BACK])
def test_refused_before_launch(call, kw):
    assert call(**kw) == c2d.EINVAL
    assert c2d.last_error() != ""


def test_single_token_calls():
    assert _rec(step=True, offsets=9 * G) == c2d.EINVAL
    assert _rec(step=True, tokens=2) == c2d.EINVAL
    assert c2d._load().gated_recurrence(None, None) == c2d.EINVAL
    assert c2d._load().gated_recurrence_backward(None, None) == c2d.EINVAL
    assert c2d._load().gated_recurrence_workspace_size(None, None) == c2d.EINVAL


@pytest.mark.parametrize("pitch,columns,ok", [(192, (0, 64, 128), True), (192, (128, 0, 64), True), (160, (0, 64, 96), False),
                                              (128, (0, 64, 128), False), (200, (0, 65, 130), True)])
def test_gradients_may_be_slices_of_one_tensor(pitch, columns, ok):
    kw = {}
    for name, c in zip(("grad_x", "grad_forget", "grad_gate"), columns):
        kw.update({name: 8 * G + 2 * c, f"{name}_token": pitch, f"{name}_batch": 100 * pitch})
    assert (_back(**kw) >= 0) == ok
    assert (_back(offsets=20 * G, **kw) >= 0) == ok


def test_slices_of_different_pitch_are_refused():
    kw = {"grad_x": 8 * G, "grad_forget": 8 * G + 128}
    kw.update(grad_x_token=192, grad_x_batch=19200, grad_forget_token=256, grad_forget_batch=25600)
    assert _back(**kw) == c2d.EINVAL


@pytest.mark.parametrize("call,kw", [(_rec, dict(tokens=1 << 30, nseq=2, x_batch=0, x_token=0)), (_rec, dict(nseq=(1 << 30) + 1)),
                                     (_rec, dict(channels=(1 << 30) + 1)), (_back, dict(tokens=(1 << 30) + 1, nseq=1)),
                                     (_back, dict(channels=(1 << 30) + 1))])
def test_too_large_is_unsupported(call, kw):
    assert call(**kw) == c2d.EUNSUPPORTED


def _wide(channels, back, **kw):
    rows = ("grad", "x", "forget", "grad_x", "grad_forget") if back else ("x", "forget", "y")
    return dict(channels=channels, tokens=1, nseq=1, gate=0, state=0, state_rows=0, **({"grad_gate": 0, "grad_state": 0} if back else {}),
                **{f"{t}_{k}": channels for t in rows for k in ("batch", "token")}, **kw)


def test_too_many_threads_are_refused_before_any_launch():
    lib = c2d._load()
    assert _rec(**_wide(1 << 30, False, dtype=c2d.DTYPE_F32)) == c2d.EUNSUPPORTED and "2^32" in c2d.last_error()
    assert _rec(step=True, **_wide(1 << 24, False, y=1 << 40) | dict(nseq=1 << 20, x_token=0, forget_token=0)) == c2d.EUNSUPPORTED
    assert "2^32" in c2d.last_error()
    lib.conv2d_set_workspace(100 * G, 1 << 45)
    try:
        # the gradient's own launches, and the bias gradient's alone
        assert _back(size=False, **_wide(1 << 30, True, dtype=c2d.DTYPE_F32)) == c2d.EUNSUPPORTED and "2^32" in c2d.last_error()
        assert _back(size=False, **_wide(1 << 28, True)) == c2d.EUNSUPPORTED and "2^32" in c2d.last_error()
    finally:
        lib.conv2d_set_workspace(None, 0)


def test_workspace_sizes():
    assert _rec(size=True) == 0  # two short sequences: not split
    one = dict(nseq=1, tokens=20000)
    assert _rec(size=True, **one) > 0
    assert _rec(size=True, nseq=0) == 0
    with_bias, without = _back(), _back(grad_forget_bias=0)
    assert with_bias - without >= 2 * D * 4  # a sum for each chunk
    assert without >= 2 * 2 * 2 * D * 4  # two numbers for each of two tiles of two sequences
    c2d._load().conv2d_set_workspace(None, 0)
    assert _back(size=False) == c2d.EUNSUPPORTED
    assert "needs a workspace" in c2d.last_error()


def test_nothing_to_do_is_fine_without_a_device():
    assert _rec(nseq=0, x=0, forget=0, y=0) == c2d.OK
    assert _rec(step=True, nseq=0, x=0, forget=0, y=0) == c2d.OK
    for tokens in (0, 1, 100, 1 << 20):
        assert _rec(nseq=0, tokens=tokens) == c2d.OK and _rec(size=True, nseq=0, tokens=tokens) == 0
        assert _back(size=False, nseq=0, tokens=tokens, grad_forget_bias=0) == c2d.OK and _back(nseq=0, tokens=tokens) == 0


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="needs a machine without a GPU")
def test_no_device_returns_ehip_not_a_crash():
    for call in (_rec, lambda: _rec(step=True), lambda: _rec(offsets=20 * G, slots=21 * G)):
        assert call() == c2d.EHIP
        assert c2d.last_error() != ""


def test_binding_refuses():
    x = torch.zeros(2, 5, 8)
    for call in (lambda: c2d.gated_recurrence(x, x), lambda: c2d.gated_recurrence_step(x[0], x[0], state=x[0]),
                 lambda: c2d.gated_recurrence_backward(x, x, x)):
        with pytest.raises(ValueError, match="expected a GPU"):
            call()
    with pytest.raises(ValueError, match="unsupported dtype"):
        c2d.gated_recurrence(x.double(), x.double())
