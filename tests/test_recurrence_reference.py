"""The 64-bit reference of the recurrence's gradient against torch's differentiation and against differences (CPU only)."""
import torch

import recurrence_reference as ref

LENGTHS = [5, 0, 1, 7]


def _case(seed, d=6):
    g = torch.Generator().manual_seed(seed)
    n = sum(LENGTHS)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    return dict(x=r(n, d), forget=r(n, d), gate=r(n, d), bias=r(d) + 1, state=r(6, d)), r(n, d), r(6, d), [4, 0, -1, 2]


def _run(c, coupled, slots):
    """The definition, differentiable: y and the final states."""
    f = torch.sigmoid(c["forget"] + c["bias"])
    state, ys, first = list(c["state"].unbind(0)), [], 0
    for i, n in enumerate(LENGTHS):
        kept = 0 <= slots[i] < len(state)
        h = state[slots[i]] if kept else torch.zeros_like(f[0])
        for t in range(first, first + n):
            h = f[t] * h + ((1 - f[t]) if coupled else 1) * c["x"][t]
            ys.append(h * c["gate"][t] * torch.sigmoid(c["gate"][t]))
        if kept:
            state[slots[i]] = h
        first += n
    return torch.stack(ys), torch.stack(state)


def _check(coupled):
    c, e, es, slots = _case(3 + coupled)
    leaves = {k: v.clone().requires_grad_() for k, v in c.items()}
    y, state = _run(leaves, coupled, slots)
    want, _, new, _, _ = ref.forward(c["x"], c["forget"], c["gate"], c["bias"], coupled, c["state"], slots, LENGTHS)
    assert torch.allclose(y, want, rtol=0, atol=1e-13) and torch.allclose(state, new, rtol=0, atol=1e-13)
    loss = (y * e).sum() + (state * es).sum()
    loss.backward()
    got = ref.backward(e, c["x"], c["forget"], c["gate"], c["bias"], coupled, c["state"], es, slots, LENGTHS)
    for name, (value, _) in zip(["x", "forget", "gate", "bias", "state"], got):
        assert torch.allclose(value, leaves[name].grad, rtol=0, atol=1e-12), name
    for name, (value, _) in zip(["x", "forget", "gate", "bias", "state"], got):  # differences along one direction
        g = torch.Generator().manual_seed(11)
        v = torch.randn(c[name].shape, generator=g, dtype=torch.float64)
        step = 1e-5
        side = []
        for s in (step, -step):
            y, state = _run({**c, name: c[name] + s * v}, coupled, slots)
            side.append((y * e).sum() + (state * es).sum())
        assert abs((side[0] - side[1]) / (2 * step) - (value * v).sum()) <= 1e-6 * (1 + value.abs().sum()), name


def test_gradient_of_the_coupled_form():
    _check(True)


def test_gradient_of_the_plain_form():
    _check(False)
