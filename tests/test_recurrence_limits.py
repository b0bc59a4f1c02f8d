"""What the recurrence's entry points ask for and refuse at the ends of their ranges, without a GPU (CPU only)."""
import random

import pytest

import test_recurrence_abi as abi


@pytest.mark.parametrize("tokens", [0, 100, 1 << 30])
@pytest.mark.parametrize("bias", [0, 11 * abi.G])
def test_gradient_of_no_sequences_needs_nothing(tokens, bias):
    """Packed rows without a sequence: no chunk, and so no workgroup that would look for its offsets."""
    assert abi._back(nseq=0, tokens=tokens, offsets=20 * abi.G, grad_forget_bias=bias) == 0


def _outs(firsts, batch, token, **kw):
    names = ("grad_x", "grad_forget", "grad_gate")
    kw = {"tokens": 10, **kw}
    for name, first in zip(names, firsts):
        kw[name] = 8 * abi.G + 2 * first
    for name, b, t in zip(names, batch if isinstance(batch, tuple) else (batch,) * 3,
                          token if isinstance(token, tuple) else (token,) * 3):
        kw.update({f"{name}_batch": b, f"{name}_token": t})
    return kw


D = abi.D


@pytest.mark.parametrize("kw", [
    _outs((0, 10 * D, 20 * D), 30 * D, D),                       # [batch, 3, tokens, channels], by the second
    _outs((20 * D, 0, 10 * D), 30 * D + 5, D),
    _outs((0, 2 * D, 4 * D), D, 6 * D),                          # tokens outside: [tokens, 3, batch, channels]
    _outs((0, D, 2 * D), 3 * D, 6 * D),                          # [tokens, batch, 3, channels]
    _outs((0, 10 * D, 35 * D), 100 * D, 3 * D),                  # rows between rows, not in order
    _outs((0, D, 2 * D), (1, 5 * D, 0), 3 * D, nseq=1),          # batch strides of a single sequence
    _outs((0, D, 2 * D), 3 * D, (0, 7 * D, 1), tokens=1),        # token strides of single tokens
])
def test_gradients_may_stand_between_each_other(kw):
    assert abi._back(**kw) >= 0, abi.c2d.last_error()


@pytest.mark.parametrize("kw", [
    _outs((0, 10 * D - 1, 20 * D), 30 * D, D),
    _outs((0, 10 * D, 20 * D + 1), 30 * D, D),                   # the last one's last row in the next entry's first
    _outs((0, 2 * D, 4 * D + 1), D, 6 * D),
    _outs((0, 3 * D, 35 * D), 100 * D, 3 * D),                   # a token later
    _outs((0, 100 * D + 9 * D, 35 * D), 100 * D, 3 * D),         # a batch entry and some tokens later
    _outs((0, 100 * D - 9 * D + 1, 35 * D), 100 * D, 3 * D),     # a batch entry later and some tokens before
    _outs((0, D, 2 * D), (30 * D, 33 * D, 30 * D), 3 * D),
    _outs((0, D, 2 * D), 60 * D, (3 * D, 4 * D, 3 * D)),
])
def test_gradients_that_share_values_are_refused(kw):
    assert abi._back(**kw) == abi.c2d.EINVAL


def test_shared_values_by_enumeration():
    """Two outputs of random equal strides are refused where some value of theirs is the same, and nowhere else."""
    r = random.Random(3)
    seen = [0, 0]
    for _ in range(3000):
        nb, nt, w = r.randint(1, 4), r.randint(1, 5), r.randint(1, 3)
        batch, token = r.randint(1, 40), r.randint(1, 24)
        first = [r.randint(0, 60) for _ in range(2)]
        cells = [[f + b * batch + t * token + c for b in range(nb) for t in range(nt) for c in range(w)] for f in first]
        want = all(len(set(c)) == len(c) for c in cells) and not set(cells[0]) & set(cells[1])
        kw = {"channels": w, "nseq": nb, "tokens": nt, "gate": 0, "grad_gate": 0}
        for name, f in zip(("grad_x", "grad_forget"), first):
            kw.update({name: 8 * abi.G + 2 * f, f"{name}_batch": batch, f"{name}_token": token})
        assert (abi._back(**kw) >= 0) <= want, (kw, first)
        simple = nb == 1 or nt == 1 or batch >= (nt - 1) * token + w or token >= (nb - 1) * batch + w
        if simple and token >= w and batch >= w:  # others are refused whether or not they share
            assert (abi._back(**kw) >= 0) == want, (kw, first)
            seen[want] += 1
    assert min(seen) > 200
