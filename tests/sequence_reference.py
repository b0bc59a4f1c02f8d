"""The sequence operators from their definitions in 64 bits, token by token on the CPU, with bounds on the error a
32-bit evaluation may have (shared by the GPU tests).

Every function takes CPU tensors and returns, next to the result, the largest error that rounding can explain. U32 =
2^-24 is the error of one 32-bit rounding, U[type] that of the one rounding to the storage type; a hardware exp2, log2
or reciprocal is counted as two roundings.
"""
import torch

U32 = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = 2.0 ** -25  # half of float16's smallest step


def silu_error(v, error):
    """Bound for silu(v) given one for v: its slope is under 1.1; exp's argument has the relative error of two
    roundings, its value, the sum, the reciprocal and the product six more."""
    return 1.1 * error + U32 * v.abs() * (2 * v.abs() + 8)


def stored(y, error, dtype):
    return error + U[dtype] * (y.abs() + error) + TINY


def activate(v, error, act, alpha=None):
    if act == "relu":
        return v.clamp(min=0), error
    if act == "silu":
        return v * torch.sigmoid(v), silu_error(v, error)
    if act == "prelu":
        a = alpha.double()
        return torch.where(v >= 0, v, a * v), error * a.abs().clamp(min=1) + U32 * (a * v).abs()
    return v, error


def conv(x, w, bias, alpha, act, state, slots, lengths, fresh):
    """x: packed rows [tokens, channels]. Returns y, its bound and the new state (exact)."""
    d, width = w.shape
    y = torch.zeros(x.shape, dtype=torch.float64)
    err = torch.zeros_like(y)
    new = None if state is None else state.clone()
    first = 0
    for i, n in enumerate(lengths):
        row = i if slots is None else int(slots[i])
        kept = state is not None and 0 <= row < state.shape[0]
        before = state[row].double() if kept and not fresh else torch.zeros(width - 1, d, dtype=torch.float64)
        line = torch.cat([before, x[first:first + n].double()])
        for t in range(n):
            terms = line[t:t + width] * w.double().t()
            v = terms.sum(0) + (0 if bias is None else bias.double())
            size = terms.abs().sum(0) + (0 if bias is None else bias.double().abs())
            y[first + t], err[first + t] = activate(v, (width + 2) * U32 * size, act, alpha)
        if kept:
            new[row] = line[n:].to(new.dtype)
        first += n
    return y, stored(y, err, x.dtype), new


def scan(u, dt, A, B, C, skip, gate, dt_bias, softplus, state, slots, lengths, fresh):
    """Packed rows; B, C [tokens, groups, states]. Returns y, its bound, the new state and its bound."""
    d, n = A.shape
    groups = B.shape[1]
    a = A.double()
    y = torch.zeros(u.shape, dtype=torch.float64)
    err = torch.zeros_like(y)
    new = None if state is None else state.double().clone()
    new_err = None if state is None else torch.zeros_like(new)
    zero = torch.zeros((), dtype=torch.float64)
    first = 0
    for i, length in enumerate(lengths):
        row = i if slots is None else int(slots[i])
        kept = state is not None and 0 <= row < state.shape[0]
        h = state[row].double() if kept and not fresh else torch.zeros(d, n, dtype=torch.float64)
        e = torch.zeros(d, n, dtype=torch.float64)
        for t in range(first, first + length):
            x = u[t].double()
            raw = dt[t].double() + (0 if dt_bias is None else dt_bias.double())
            if softplus:
                step = torch.logaddexp(raw, zero)
                # the sum's rounding and exp's argument: relative errors |raw| and 2 |raw|; the rest: eight roundings
                rel = 3 * raw.abs() + 8
            else:
                step, rel = raw, torch.ones_like(raw)
            b = B[t].double().repeat_interleave(d // groups, 0)
            c = C[t].double().repeat_interleave(d // groups, 0)
            power = step[:, None] * a
            decay = torch.exp(power)
            add = (step * x)[:, None] * b
            before = h
            h = decay * before + add
            # the exponent's own relative error: step's, A's scale to base two (two roundings), the product's; exp2: two
            e = decay * e + U32 * ((2 + (3 + rel[:, None]) * power.abs()) * (decay * before).abs()
                                   + (3 + rel[:, None]) * add.abs() + h.abs())
            s = (h * c).sum(-1)
            es = (e * c.abs()).sum(-1) + (n + 2) * U32 * (h * c).abs().sum(-1)
            if skip is not None:
                s = s + skip.double() * x
                es = es + U32 * ((skip.double() * x).abs() + s.abs())
            if gate is not None:
                g = gate[t].double()
                z = g * torch.sigmoid(g)
                es = es * z.abs() + s.abs() * silu_error(g, 0) + U32 * (s * z).abs()
                s = s * z
            y[t], err[t] = s, es
        if kept:
            new[row], new_err[row] = h, e
        first += length
    return y, stored(y, err, u.dtype), new, new_err


def w4(x, codes, scales, zeros, group, bias, alpha, residual, act, before):
    """x [rows, in]. Sums of 32-bit products, in any order of at most in / 32 + 64 dependent additions; a code may be
    taken with an offset of at most 31 that is subtracted again."""
    k = x.shape[1]
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(1)[:, :k].double()
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(group, 1)[:, :k]
    s = scales.double().repeat_interleave(group, 1)[:, :k]
    xd = x.double()
    v = xd @ ((q - z) * s).t()
    size = xd.abs() @ s.abs().t() * (31 + 24)
    err = U32 * (k / 32 + 64) * size
    if bias is not None:
        v = v + bias.double()
    r = 0 if residual is None else residual.double()
    if before:
        v = v + r
    err = err + 2 * U32 * (v.abs() + (0 if bias is None else bias.double().abs()))
    y, err = activate(v, err, act, alpha)
    if not before:
        y = y + r
    err = err + U32 * y.abs()
    return y, stored(y, err, x.dtype)


def close(got, want, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)}, expected {tuple(want.shape)}"
    assert torch.isfinite(got).all(), f"{what}: not finite"
    off = (got - want).abs()
    bad = off > bound
    if bad.any():
        at = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {at}: got {float(got[at])}, "
                             f"expected {float(want[at])} within {float(bound[at])}")
