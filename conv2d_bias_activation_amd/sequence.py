"""Sequence operators of the library (include/sequence_ops.h): the short causal convolution
and the selective state space scan, for prompts and for single tokens, and products of a few
token rows with 4-bit weights.

As in the rest of the binding, PyTorch supplies device memory and streams, and everything is
computed by the library's HIP kernels; this module checks tensors, fills the C structs and
allocates outputs. Activations are channel-last, and a tensor may be a slice of a wider one
(the columns of one projection), as long as the channels of a token are contiguous. ``out`` may
be a slice too, but not of a tensor that holds an input: from its first to its last value it may
not overlap one.

A call on ``stream`` enqueues its work there (default: the device's current stream) and
allocates what it returns there too; inputs made on another stream have to be waited for by
the caller, as with any kernel.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _ACTS, _DTYPES, RES_BEFORE_ACT, _check, _load, _use_workspace, _ws_cache, _ws_key

__all__ = ["causal_conv1d", "causal_conv1d_step", "selective_scan", "selective_scan_step", "w4_pack", "matvec_w4",
           "W4Weights"]

# struct causal_conv1d_args, selective_scan_args and matvec_w4_args, field by field
_CONV = struct.Struct("@8P5q7i0q")
_SCAN = struct.Struct("@12P14q8i0q")
_W4 = struct.Struct("@6P3q7i0q")


def _stream_handle(index):
    return torch.cuda.current_stream(index).cuda_stream


# the current stream's handle and the current device, without what torch.cuda puts around them
# (a tensor on the GPU has initialised it); a torch without the private names takes the public way
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_handle)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(name, args, device, stream):
    """The entry point `name` on packed args, on `stream`, with the tensors' device current."""
    fn = getattr(_load(), name)
    handle = _raw_stream(device.index) if stream is None else stream.cuda_stream
    if device.index == _current_device():
        rc = fn(args, handle)
    else:
        with torch.cuda.device(device):
            rc = fn(args, handle)
    if rc:
        _check(rc)


def _new(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):  # so that the allocator reuses the memory after this stream's work
        return torch.empty(shape, dtype=dtype, device=device)


def _new_like(x, stream):
    if stream is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    with torch.cuda.stream(stream):
        return torch.empty_like(x, memory_format=torch.contiguous_format)


def _scratch(device, stream, workspace, need):
    """Registers the workspace of a call."""
    if workspace is None and device.index == _current_device():
        ws = _ws_cache.get(_ws_key(device.index, _raw_stream(device.index) if stream is None else stream.cuda_stream))
        if ws is not None and ws.numel() >= need:  # as below, without the detours
            _check(_load().conv2d_set_workspace(ws.data_ptr(), ws.numel()))
            return
    _use_workspace(device, torch.cuda.current_stream(device) if stream is None else stream, workspace, need)


def _fail(name, what):
    raise ValueError(f"{name} {what}")


def _refuse(name, t, shape, dtype, device):
    if t.shape != shape:
        _fail(name, f"must have shape {tuple(shape)}, has {tuple(t.shape)}")
    if t.dtype != dtype:
        _fail(name, f"has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        _fail(name, f"is on {t.device}, expected {device}")


def _rows(name, t, shape, dtype, device):
    """Checks token rows (any strides but the last); their address."""
    if t.shape != shape or t.dtype != dtype or t.device != device:
        _refuse(name, t, shape, dtype, device)
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        _fail(name, "must have the values of a token contiguous")
    return t.data_ptr()


def _dense(name, t, shape, dtype, device):
    """Checks a contiguous tensor or None; its address."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype != dtype or t.device != device:
        _refuse(name, t, shape, dtype, device)
    if not t.is_contiguous():
        _fail(name, "must be contiguous")
    return t.data_ptr()


def _storage(t, name="x"):
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {t.dtype}")
    if not t.is_cuda:
        _fail(name, f"is on {t.device}, expected a GPU")
    return dt


def _geometry(x, seq_offsets, step, name="x"):
    """(sequences, tokens, batch stride, token stride) of token rows x."""
    if step or seq_offsets is not None:
        if x.dim() != 2:
            _fail(name, "must be [sequences, channels]" if step else "must be [tokens, channels] with seq_offsets")
        if step:
            return x.shape[0], 1, 0, x.stride(0)
        if seq_offsets.dim() != 1 or seq_offsets.shape[0] < 1:
            _fail("seq_offsets", "must be [sequences + 1]")
        return seq_offsets.shape[0] - 1, x.shape[0], 0, x.stride(0)
    if x.dim() != 3:
        _fail(name, "must be [batch, tokens, channels], or [tokens, channels] with seq_offsets")
    return x.shape[0], x.shape[1], x.stride(0), x.stride(1)


def _state_rows(state, shape, dtype, device):
    if state is None:
        return 0, 0
    if state.dim() != len(shape) + 1:
        _fail("state", f"must be [rows, {', '.join(map(str, shape))}]")
    return _dense("state", state, (state.shape[0], *shape), dtype, device), state.shape[0]


def _act(act):
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(_ACTS)}, got {act!r}")
    return code


def _conv(name, x, w, bias, alpha, act, state, slots, fresh, seq_offsets, out, stream, step):
    dt = _storage(x)
    dev, dtype, shape = x.device, x.dtype, x.shape
    nseq, tokens, x_batch, x_token = _geometry(x, seq_offsets, step)
    channels = shape[-1]
    if w.dim() != 2 or w.shape[0] != channels:
        _fail("w", f"must be [{channels}, width]")
    width = w.shape[1]
    xp = _rows("x", x, shape, dtype, dev)
    wp = _dense("w", w, w.shape, dtype, dev)
    bp = _dense("bias", bias, (channels,), torch.float32, dev)
    ap = _dense("alpha", alpha, (channels,), torch.float32, dev)
    sp, rows = _state_rows(state, (width - 1, channels), dtype, dev)
    op = _dense("seq_offsets", seq_offsets, (nseq + 1,), torch.int32, dev)
    lp = _dense("slots", slots, (nseq,), torch.int32, dev)
    if out is None:
        out = _new_like(x, stream)
        yp, y_batch, y_token = out.data_ptr(), tokens * channels, channels
    else:
        yp = _rows("out", out, shape, dtype, dev)
        y_batch, y_token = (out.stride(0), out.stride(1)) if len(shape) == 3 else (0, out.stride(0))
    _call(name, _CONV.pack(xp, wp, bp, ap, sp, yp, op, lp, x_batch, x_token, y_batch, y_token, tokens, nseq, rows,
                           channels, width, _act(act), dt, 1 if fresh else 0), dev, stream)
    return out


def causal_conv1d(x, w, bias=None, alpha=None, *, act="none", state=None, slots=None, fresh=False, seq_offsets=None,
                  out=None, stream=None):
    """y[t, c] = act(bias[c] + sum_j w[c, j] * x[t - (width - 1) + j, c]) along each sequence.

    x: [batch, tokens, channels], or with ``seq_offsets`` (int32 [sequences + 1] on the GPU) the
    sequences packed as [tokens, channels]; float32, bfloat16 or float16, any strides but the
    last. w: [channels, width], width 2 to 4, in x's dtype. bias, alpha (the slopes of
    act="prelu"): float32 [channels]. ``state`` [rows, width - 1, channels] in x's dtype holds
    the inputs before a sequence's first and is updated in place to its last ones; sequence i
    uses row slots[i] (int32, default i; a slot outside the rows: no state). ``fresh``: the
    sequences start from zeros and the state is only written. Returns y, shaped as x."""
    return _conv("causal_conv1d", x, w, bias, alpha, act, state, slots, fresh, seq_offsets, out, stream, False)


def causal_conv1d_step(x, w, bias=None, alpha=None, *, state, act="none", slots=None, out=None, stream=None):
    """causal_conv1d for one token of each sequence: x [sequences, channels]."""
    return _conv("causal_conv1d_step", x, w, bias, alpha, act, state, slots, False, None, out, stream, True)


def _scan(name, u, dt, A, B, C, skip, gate, dt_bias, softplus, state, slots, fresh, seq_offsets, longest, out, stream,
          workspace, step):
    code = _storage(u, "u")
    dev, dtype, shape = u.device, u.dtype, u.shape
    nseq, tokens, _, u_token = _geometry(u, seq_offsets, step, "u")
    channels = shape[-1]
    if A.dim() != 2 or A.shape[0] != channels:
        _fail("A", f"must be [{channels}, states]")
    states = A.shape[1]
    if B.dim() != u.dim() + 1 or B.shape[-2] < 1:
        _fail("B", "must have u's leading dimensions, then [groups, states]")
    groups = B.shape[-2]
    bc = (*shape[:-1], groups, states)
    up = _rows("u", u, shape, dtype, dev)
    dp = _rows("dt", dt, shape, dtype, dev)
    bp = _rows("B", B, bc, dtype, dev)
    cp = _rows("C", C, bc, dtype, dev)
    if groups > 1 and (B.stride(-2) != states or C.stride(-2) != states):
        _fail("B and C", "must have the groups of a token contiguous")
    gp = 0 if gate is None else _rows("gate", gate, shape, dtype, dev)
    Ap = _dense("A", A, A.shape, torch.float32, dev)
    kp = _dense("skip", skip, (channels,), torch.float32, dev)
    tp = _dense("dt_bias", dt_bias, (channels,), torch.float32, dev)
    sp, rows = _state_rows(state, (channels, states), torch.float32, dev)
    op = _dense("seq_offsets", seq_offsets, (nseq + 1,), torch.int32, dev)
    lp = _dense("slots", slots, (nseq,), torch.int32, dev)
    if out is None:
        out = _new_like(u, stream)
        yp = out.data_ptr()
    else:
        yp = _rows("out", out, shape, dtype, dev)
    if len(shape) == 3:
        strides = (*u.stride()[:2], *dt.stride()[:2], *B.stride()[:2], *C.stride()[:2],
                   *((0, 0) if gate is None else gate.stride()[:2]), *out.stride()[:2])
    else:
        strides = (0, u_token, 0, dt.stride(0), 0, B.stride(0), 0, C.stride(0), 0, 0 if gate is None else gate.stride(0),
                   0, out.stride(0))
    args = _SCAN.pack(up, dp, Ap, bp, cp, kp, gp, tp, sp, yp, op, lp, *strides, tokens, longest or 0, nseq, rows, channels,
                      groups, states, 1 if softplus else 0, code, 1 if fresh else 0)
    if not step:
        need = 0
        if workspace is None:
            size = ctypes.c_size_t(0)
            _check(_load().selective_scan_workspace_size(args, ctypes.byref(size)))
            need = size.value
        if need or workspace is not None:
            _scratch(dev, stream, workspace, need)
    _call(name, args, dev, stream)
    return out


def selective_scan(u, dt, A, B, C, *, skip=None, gate=None, dt_bias=None, softplus=False, state=None, slots=None,
                   fresh=False, seq_offsets=None, longest=None, out=None, stream=None, workspace=None):
    """Selective state space scan along each sequence. With d = dt + dt_bias (through
    log(1 + exp(d)) with ``softplus``), h the [channels, states] state and g a channel's group:

        h[c, n] = exp(d[t, c] * A[c, n]) * h[c, n] + d[t, c] * u[t, c] * B[t, g, n]
        y[t, c] = (sum_n h[c, n] * C[t, g, n] + skip[c] * u[t, c]) * silu(gate[t, c])

    u, dt, gate: [batch, tokens, channels], or packed [tokens, channels] with ``seq_offsets``
    (int32 [sequences + 1] on the GPU); B, C: the same leading dimensions, then [groups, states];
    all of one dtype (float32, bfloat16 or float16), any strides before the last. A [channels,
    states], skip and dt_bias [channels]: float32. ``state`` float32 [rows, channels, states] is
    read and updated in place; ``slots`` and ``fresh`` as for causal_conv1d. ``longest``: tokens
    of the longest packed sequence where known; it only steers how the work is split. A split
    call keeps its chunks' states in the workspace (``workspace`` as everywhere in the binding;
    False: never split; inside a graph capture pass a tensor that lives as long as the graph).
    Returns y, shaped as u."""
    return _scan("selective_scan", u, dt, A, B, C, skip, gate, dt_bias, softplus, state, slots, fresh, seq_offsets,
                 longest, out, stream, workspace, False)


def selective_scan_step(u, dt, A, B, C, *, state, skip=None, gate=None, dt_bias=None, softplus=False, slots=None,
                        out=None, stream=None):
    """selective_scan for one token of each sequence: u [sequences, channels], B [sequences, groups, states]."""
    return _scan("selective_scan_step", u, dt, A, B, C, skip, gate, dt_bias, softplus, state, slots, False, None, None,
                 out, stream, False, True)


class W4Weights:
    """4-bit weights laid out by w4_pack for matvec_w4 (``data``: the packed bytes)."""
    __slots__ = ("data", "in_features", "out_features", "group", "zeros", "dtype", "device")

    def __init__(self, data, in_features, out_features, group, zeros, dtype):
        self.data, self.in_features, self.out_features = data, in_features, out_features
        self.group, self.zeros, self.dtype, self.device = group, zeros, dtype, data.device


def w4_pack(codes, scales, zeros=None, *, in_features=None, group=128, stream=None):
    """Lays out 4-bit weights once for matvec_w4. Weight (o, k) is (code - zero) * scale.

    codes: uint8 [out_features, ceil(in_features / 2)], the even input's code in the low half;
    in_features defaults to twice its columns. scales: bfloat16 or float16 [out_features,
    ceil(in_features / group)], in the dtype of the activations; zeros: uint8 of the same shape
    (0 to 15), default 8. group: 32, 64 or 128 inputs."""
    if codes.dim() != 2:
        _fail("codes", "must be [out_features, ceil(in_features / 2)]")
    n, k = codes.shape[0], 2 * codes.shape[1] if in_features is None else int(in_features)
    if scales.dtype not in (torch.bfloat16, torch.float16):
        _fail("scales", f"has dtype {scales.dtype}, expected bfloat16 or float16")
    dt = _storage(scales, "scales")
    dev = codes.device
    lib = _load()
    nbytes = ctypes.c_size_t(0)
    _check(lib.matvec_w4_packed_bytes(n, k, group, 0 if zeros is None else 1, ctypes.byref(nbytes)))
    groups = -(-k // group)
    cp = _dense("codes", codes, (n, (k + 1) // 2), torch.uint8, scales.device)
    sp = _dense("scales", scales, (n, groups), scales.dtype, dev)
    zp = _dense("zeros", zeros, (n, groups), torch.uint8, dev)
    data = _new((nbytes.value,), torch.uint8, dev, stream)
    with torch.cuda.device(dev):
        _check(lib.matvec_w4_pack(cp, sp, zp, data.data_ptr(), n, k, group, dt,
                                   _raw_stream(dev.index) if stream is None else stream.cuda_stream))
    return W4Weights(data, k, n, group, zeros is not None, scales.dtype)


def matvec_w4(x, weights, bias=None, alpha=None, residual=None, *, act="none", res_before_act=False, out=None,
              stream=None):
    """y = epilogue(x @ W^T) with 4-bit weights from w4_pack, for a few token rows.

    x [rows, in_features], residual [rows, out_features] in the weights' dtype, rows at any
    stride; bias, alpha (act="prelu"): float32 [out_features]. The epilogue is conv2d_fused's.
    Sums are fp32. Returns y [rows, out_features]."""
    dt = _storage(x)
    dev, dtype = weights.device, weights.dtype
    if x.dim() != 2:
        _fail("x", "must be [rows, in_features]")
    rows, n = x.shape[0], weights.out_features
    xp = _rows("x", x, (rows, weights.in_features), dtype, dev)
    bp = _dense("bias", bias, (n,), torch.float32, dev)
    ap = _dense("alpha", alpha, (n,), torch.float32, dev)
    rp = 0 if residual is None else _rows("residual", residual, (rows, n), dtype, dev)
    if out is None:
        out = _new((rows, n), dtype, dev, stream)
        yp = out.data_ptr()
    else:
        yp = _rows("out", out, (rows, n), dtype, dev)
    _call("matvec_w4", _W4.pack(xp, weights.data.data_ptr(), bp, ap, rp, yp, x.stride(0),
                                0 if residual is None else residual.stride(0), out.stride(0), rows,
                                weights.in_features, n, weights.group, 1 if weights.zeros else 0,
                                _act(act) | (RES_BEFORE_ACT if res_before_act else 0), dt), dev, stream)
    return out
