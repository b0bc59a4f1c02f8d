"""The recurrence's gates where they are all but shut or open, on the GPU against their definition in 64 bits."""
import pytest
import torch

import recurrence_reference as rec
import sequence_reference as ref

pytestmark = pytest.mark.gpu

c2d = pytest.importorskip("conv2d_bias_activation_amd")
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _gate(v, bias=None):
    """sigmoid of z = v + bias, one minus it, and bounds on their relative errors by |z| alone. The sum is off by U32 |z|; the
    argument of exp2 is z times a constant off by half a rounding, rounded once: 1.5 U32 |z| in z. exp2 adds two
    roundings, which the gate takes with the slope of the other one; the sum 1 + t and its reciprocal make three, the
    product for the other gate one more. A gate below the smallest normal number may be zero."""
    z = v.double() + (torch.zeros(v.shape[-1], dtype=torch.float64) if bias is None else bias.double())
    f, k = torch.sigmoid(z), torch.sigmoid(-z)
    arg, tiny = 2.5 * z.abs() + 2, 2.0 ** -126
    return (f, k, ref.U32 * (arg * k + 3) * 1.001 + tiny / f.clamp(min=1e-300),
            ref.U32 * (arg * f + 4) * 1.001 + tiny / k.clamp(min=1e-300))


def _on(t):
    return None if t is None else t.to(DEV)


def _check(monkeypatch, kind, lengths, v, bias, coupled, seed):
    """Prompts, tokens and gradients whose forget logits are v, one for each channel, at every token."""
    monkeypatch.setattr(rec, "_gate", _gate)
    g = torch.Generator().manual_seed(seed)
    dtype, n, d, seqs = TYPES[kind], sum(lengths), len(v), len(lengths)
    normal = lambda *s, dtype=dtype: torch.randn(*s, generator=g).to(dtype)
    x, gate, grad = normal(n, d), normal(n, d), normal(n, d)
    forget = v.to(dtype).expand(n, d).contiguous()
    state, grad_state = (normal(seqs, d, dtype=torch.float32) for _ in range(2))
    want, bound, new, new_bound, _ = rec.forward(x, forget, gate, bias, coupled, state, None, lengths)
    back = rec.backward(grad, x, forget, gate, bias, coupled, state, grad_state, None, lengths)
    kw = {"gate": _on(gate), "forget_bias": _on(bias), "coupled": coupled}
    packed = {**kw, "seq_offsets": torch.tensor([0] + lengths).cumsum(0).to(torch.int32).to(DEV), "longest": max(lengths)}
    for workspace in (None, False):
        s = _on(state.clone())
        y = c2d.gated_recurrence(_on(x), _on(forget), state=s, workspace=workspace, **packed)
        ref.close(y, want, bound, "prompt")
        ref.close(s, new, new_bound, "its state")
    gs = _on(grad_state.clone())
    got = c2d.gated_recurrence_backward(_on(grad), _on(x), _on(forget), state=_on(state), grad_state=gs, **packed)
    for name, t, (value, limit) in zip(("x", "forget", "gate", "bias", "state"), [*got, gs], back):
        if t is not None:
            ref.close(t, value, limit, f"gradient of {name}")
    first = [sum(lengths[:i]) for i in range(seqs)]
    want, bound, new, new_bound, _ = rec.forward(x[first], forget[first], gate[first], bias, coupled, state, None, [1] * seqs)
    s = _on(state.clone())
    kw["gate"] = kw["gate"][first]
    y = c2d.gated_recurrence_step(_on(x[first]), _on(forget[first]), state=s, **kw)
    ref.close(y, want, bound, "token")
    ref.close(s, new, new_bound, "its state")


ENDS = torch.cat([torch.arange(-95, -79.75, 0.25), torch.arange(80, 95.25, 0.25)])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("coupled", [True, False])
@pytest.mark.parametrize("bias", [None, 0.5, -3.0])
def test_gates_next_to_their_ends(monkeypatch, kind, coupled, bias):
    """Logits past 87, where a gate leaves the normal numbers: the other one is 1."""
    b = None if bias is None else torch.full((len(ENDS),), bias)
    _check(monkeypatch, kind, [70, 1, 600], ENDS if bias is None else ENDS - bias, b, coupled, 1)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("coupled", [True, False])
def test_logits_and_biases_that_cancel(monkeypatch, kind, coupled):
    """The gate goes by the sum alone, however large its two terms are."""
    g = torch.Generator().manual_seed(5)
    size = torch.cat([torch.tensor([100.0]).expand(40), torch.tensor([1000.0]).expand(40), torch.tensor([1e4]).expand(20)])
    v = torch.cat([(torch.rand(100, generator=g) * 2 - 1) * size,
                   torch.tensor([100.0, -100.0, 5e4, 2.3e38, 2.5e38, -2.5e38, 3e38, -3e38])])
    if kind == "f16":
        v = v.clamp(-6e4, 6e4)
    v = v.to(TYPES[kind]).float()
    bias = torch.randn(len(v), generator=g) * 2 - v
    bias[100:] = -v[100:]
    _check(monkeypatch, kind, [70, 1, 600], v, bias, coupled, 2)
