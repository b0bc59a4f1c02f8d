"""The gated linear recurrence and its gradient from their definitions in 64 bits, token by token on the CPU, with
bounds on the error a 32-bit evaluation may have.

U32 = 2^-24 is the error of one 32-bit rounding. The argument of a gate's exp2 is -log2(e) v + (-log2(e) bias), where
the rounded constant is off by half a rounding, the second product by one more, and the sum by one: in z = v + bias
that is U32 (|v| / 2 + 3 |bias| / 2 + |z|). exp2 adds two, relatively; the gate's logarithm has the slope of the other
gate in it. The sum 1 + t and the reciprocal make three, the product for the other gate one more. ``m`` bounds the sizes of the terms that make up a state or a carried gradient, which any order of joining
runs of tokens adds up; four roundings a token cover the products and sums of such an order.
"""
import torch

from sequence_reference import U, U32, silu_error
from sequence_reference import stored as _rounded


def stored(y, error, dtype):
    """With the rounding to the storage type; none for 64-bit inputs."""
    return _rounded(y, error, dtype) if dtype in U else error


def _gate(v, bias=None):
    """sigmoid of the sum, one minus it, and their relative errors."""
    b = torch.zeros(v.shape[-1], dtype=torch.float64) if bias is None else bias.double()
    v = v.double()
    z = v + b
    f, k = torch.sigmoid(z), torch.sigmoid(-z)
    arg = v.abs() / 2 + 1.5 * b.abs() + z.abs() + 2
    return f, k, U32 * (arg * k + 3) * 1.001, U32 * (arg * f + 4) * 1.001


def _start(state, slots, i, d, fresh=False):
    row = i if slots is None else int(slots[i])
    kept = state is not None and 0 <= row < state.shape[0]
    return row, kept, state[row].double() if kept and not fresh else torch.zeros(d, dtype=torch.float64)


def forward(x, forget, gate, bias, coupled, state, slots, lengths, fresh=False):
    """Packed rows. Returns y, its bound, the new state and its bound, and each token's state, size and error with those
    before it (for the gradient)."""
    tokens, d = x.shape
    xd = x.double()
    f, k, rf, rk = _gate(forget, bias)
    b = k * xd if coupled else xd
    rb = (rk if coupled else 0 * rk) + 2 * U32
    new = None if state is None else state.double().clone()
    new_err = None if state is None else torch.zeros_like(new)
    h, m, e = (torch.zeros(tokens, d, dtype=torch.float64) for _ in range(3))
    hb, mb, eb = (torch.zeros(tokens, d, dtype=torch.float64) for _ in range(3))
    first = 0
    for i, n in enumerate(lengths):
        row, kept, hc = _start(state, slots, i, d, fresh)
        mc, ec = hc.abs(), torch.zeros(d, dtype=torch.float64)
        for t in range(first, first + n):
            hb[t], mb[t], eb[t] = hc, mc, ec
            m2 = f[t] * mc + b[t].abs()
            ec = f[t] * ec + rf[t] * f[t] * mc + rb[t] * b[t].abs() + 4 * U32 * m2
            hc, mc = f[t] * hc + b[t], m2
            h[t], m[t], e[t] = hc, mc, ec
        if kept:
            new[row], new_err[row] = hc, ec
        first += n
    y, err = h, e
    if gate is not None:
        g = gate.double()
        z = g * torch.sigmoid(g)
        y = h * z
        err = e * z.abs() + h.abs() * silu_error(g, 0) + U32 * y.abs()
    return y, stored(y, err, x.dtype), new, new_err, (h, m, e, hb, mb, eb)


def backward(grad, x, forget, gate, bias, coupled, state, grad_state, slots, lengths):
    """Packed rows. Returns pairs of value and bound: grad_x, grad_forget, grad_gate, grad_forget_bias, grad_state."""
    tokens, d = x.shape
    h, m, e, hb, mb, eb = forward(x, forget, gate, bias, coupled, state, slots, lengths)[4]
    xd, ed = x.double(), grad.double()
    f, k, rf, rk = _gate(forget, bias)
    part, part_err = ed, torch.zeros_like(ed)
    dgate = dgate_err = None
    if gate is not None:
        g = gate.double()
        on, off, ron, roff = _gate(g)
        part = ed * g * on
        part_err = ed.abs() * silu_error(g, 0) + 2 * U32 * part.abs()
        slope = on * (1 + g * off)
        slope_err = (ron + 3 * U32) * slope.abs() + on * (roff + 2 * U32) * (g * off).abs() + U32 * on
        dgate = ed * h * slope
        dgate_err = stored(dgate, ed.abs() * (e * slope.abs() + h.abs() * slope_err) + 3 * U32 * dgate.abs(), x.dtype)
    G, M, E = (torch.zeros(tokens, d, dtype=torch.float64) for _ in range(3))
    new = None if grad_state is None else grad_state.double().clone()
    new_err = None if grad_state is None else torch.zeros_like(new)
    first = 0
    for i, n in enumerate(lengths):
        row, kept, c = _start(grad_state, slots, i, d)
        mc, ec = c.abs(), torch.zeros(d, dtype=torch.float64)
        for t in reversed(range(first, first + n)):
            G[t], M[t] = part[t] + c, part[t].abs() + mc
            E[t] = part_err[t] + ec + 4 * U32 * M[t]
            c, mc = f[t] * G[t], f[t] * M[t]
            ec = f[t] * E[t] + (rf[t] + 4 * U32) * mc
        if kept:
            new[row], new_err[row] = c, ec
        first += n
    dx, dx_err = (G * k, E * k + M * k * (rk + 2 * U32)) if coupled else (G, E)
    diff, diff_err = (hb - xd, eb + U32 * (mb + xd.abs())) if coupled else (hb, eb)
    w = f * k
    df = G * w * diff
    df_err = w * (E * diff.abs() + M * (diff_err + (rf + rk + 5 * U32) * diff.abs()))
    db = df.sum(0)
    db_err = df_err.sum(0) + tokens * U32 * df.abs().sum(0)
    return ((dx, stored(dx, dx_err, x.dtype)), (df, stored(df, df_err, x.dtype)), (dgate, dgate_err), (db, db_err),
            (new, new_err))
