"""Causal convolution, selective scan and 4-bit products on the GPU against their definitions in 64 bits."""
import pytest
import torch

import sequence_reference as ref

pytestmark = pytest.mark.gpu

c2d = pytest.importorskip("conv2d_bias_activation_amd")
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _rng(seed):
    return torch.Generator().manual_seed(seed)


def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def _offsets(lengths):
    return torch.tensor([0] + lengths).cumsum(0).to(torch.int32).to(DEV)


def _wide(t, extra=0, shift=0):
    """The same values on the GPU as columns of a wider tensor, `shift` values in."""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + extra + shift), float("nan"), dtype=t.dtype, device=DEV)
    view = wide[..., shift:shift + t.shape[-1]]
    view.copy_(t)
    return view


# ---------------------------------------------------------------- causal convolution

CONV = [  # type, lengths, packed, channels, width, act, what else
    ("f32", [1], False, 1, 4, "silu", {}),
    ("bf16", [77], False, 512, 4, "silu", {}),
    ("f16", [16, 16], False, 64, 4, "silu", {"slots": [2, 0]}),
    ("bf16", [33, 33, 33], False, 72, 3, "relu", {"wide": 8}),
    ("f16", [5], False, 40, 2, "prelu", {"wide": 3, "shift": 1}),
    ("f32", [130, 0, 1, 2, 3, 4, 15, 16, 17], True, 36, 4, "silu", {"slots": [8, 3, 1, 0, 5, 4, 2, 6, 7]}),
    ("bf16", [0, 0, 31, 1, 0, 48, 2], True, 1032, 4, "none", {"slots": [0, 1, 2, 3, 4, 5, 6], "wide": 1032}),
    ("f16", [7, 64, 9], True, 13, 3, "silu", {"slots": [1, -1, 5]}),
    ("bf16", [3, 20], True, 264, 4, "silu", {"state": False}),
    ("f32", [1, 0, 40], True, 129, 2, "none", {"bias": False, "fresh": True}),
    ("bf16", [2, 0, 300], True, 128, 4, "silu", {"fresh": True, "wide": 64}),
    ("bf16", [2500, 3, 2601, 0], True, 1024, 4, "silu", {"slots": [3, 2, 1, 0]}),
    ("f16", [8203], False, 1003, 3, "silu", {}),
]


def _conv_case(seed, kind, lengths, packed, d, width, act, more):
    g = _rng(seed)
    dtype = TYPES[kind]
    tokens = sum(lengths)
    c = {"x": _normal(g, tokens, d, dtype=dtype), "w": _normal(g, d, width, dtype=dtype, scale=width ** -0.5),
         "bias": _normal(g, d, scale=0.1) if more.get("bias", True) else None,
         "alpha": torch.rand(d, generator=g) if act == "prelu" else None,
         "slots": torch.tensor(more["slots"], dtype=torch.int32) if "slots" in more else None}
    rows = len(lengths) + 2
    c["state"] = _normal(g, rows, width - 1, d, dtype=dtype) if more.get("state", True) else None
    return c


def _on(t):
    return None if t is None else t.to(DEV)


@pytest.mark.parametrize("i", range(len(CONV)))
def test_conv_prompt(i):
    kind, lengths, packed, d, width, act, more = CONV[i]
    c = _conv_case(i, *CONV[i])
    fresh = more.get("fresh", False)
    want, bound, state = ref.conv(c["x"], c["w"], c["bias"], c["alpha"], act, c["state"], c["slots"], lengths, fresh)
    x = c["x"] if packed else c["x"].reshape(len(lengths), lengths[0], d)
    x = _wide(x, more.get("wide", 0), more.get("shift", 0))
    dev_state = _on(c["state"])
    if fresh and dev_state is not None:
        dev_state.fill_(float("nan"))  # it may hold anything
        state[len(lengths):] = float("nan")
    got = c2d.causal_conv1d(x, _on(c["w"]), _on(c["bias"]), _on(c["alpha"]), act=act, state=dev_state,
                            slots=_on(c["slots"]), fresh=fresh, seq_offsets=_offsets(lengths) if packed else None)
    assert got.shape == x.shape
    ref.close(got.reshape(-1, d), want, bound, f"conv {CONV[i]}")
    if dev_state is not None:
        assert torch.equal(dev_state.cpu().nan_to_num(7.5), state.nan_to_num(7.5)), "state"


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,d,width,act", [(1, 1, 2, "none"), (1, 2048, 4, "silu"), (9, 264, 3, "relu"), (5, 77, 4, "silu"),
                                              (3, 40, 2, "prelu")])
def test_conv_token(kind, rows, d, width, act):
    c = _conv_case(rows + d, kind, [1] * rows, True, d, width, act, {})
    slots = torch.randperm(rows + 2, generator=_rng(1))[:rows].to(torch.int32)
    if rows > 4:
        slots[2], slots[3] = -1, rows + 2  # rows without a state
    want, bound, state = ref.conv(c["x"], c["w"], c["bias"], c["alpha"], act, c["state"], slots, [1] * rows, False)
    dev_state = _on(c["state"])
    got = c2d.causal_conv1d_step(_wide(c["x"], d), _on(c["w"]), _on(c["bias"]), _on(c["alpha"]), act=act, state=dev_state,
                                 slots=_on(slots))
    ref.close(got, want, bound, "conv token")
    assert torch.equal(dev_state.cpu(), state)


def test_conv_of_a_large_batch_is_that_of_its_sequences():
    """A batch past the size where runs grow longest has the bits of its sequences convolved one by one."""
    d, lengths = 4096, [1000, 17, 3000, 1, 0, 5000, 2500, 4999]
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn(sum(lengths), d, generator=g, device=DEV).bfloat16()
    w = torch.randn(d, 4, generator=g, device=DEV).bfloat16()
    state = torch.randn(len(lengths), 3, d, generator=g, device=DEV).bfloat16()
    alone = state.clone()
    y = c2d.causal_conv1d(x, w, act="silu", state=state, seq_offsets=_offsets(lengths))
    first = 0
    for i, n in enumerate(lengths):
        for part in range(0, n, 1000):
            cut = x[first + part:first + min(n, part + 1000)]
            z = c2d.causal_conv1d(cut[None], w, act="silu", state=alone[i:i + 1])
            assert torch.equal(z[0], y[first + part:first + part + len(cut)])
        first += n
    assert torch.equal(state, alone)


# ---------------------------------------------------------------- selective scan

SCAN = [  # type, lengths, packed, channels, states, groups, what else
    ("f32", [1], False, 1, 1, 1, {}),
    ("f32", [37], False, 64, 16, 1, {}),
    ("bf16", [50, 50], False, 96, 16, 1, {"slots": [3, 1]}),
    ("f16", [17], False, 240, 64, 2, {"wide": 16}),
    ("bf16", [33, 0, 1, 2, 70, 16], True, 130, 16, 1, {"slots": [0, 1, 2, 3, 4, 5], "wide": 130}),
    ("f16", [0, 65, 1, 0], True, 60, 5, 3, {"slots": [5, -1, 2, 0]}),
    ("f32", [20, 19], True, 36, 100, 4, {"wide": 1, "shift": 1}),
    ("bf16", [9], True, 16, 256, 1, {"state": False}),
    ("f32", [0, 40, 1], True, 65, 24, 1, {"fresh": True}),
    ("bf16", [128], False, 64, 16, 1, {"plain": True}),
    ("f16", [900], False, 64, 16, 1, {}),
    ("bf16", [1500, 3, 700], True, 72, 16, 1, {"wide": 8}),
    ("f32", [1100], True, 40, 33, 2, {}),
]


def _scan_case(seed, kind, lengths, d, n, groups, more):
    g = _rng(seed)
    dtype = TYPES[kind]
    tokens = sum(lengths)
    c = {"u": _normal(g, tokens, d, dtype=dtype), "dt": _normal(g, tokens, d, dtype=dtype, scale=0.5),
         "A": -torch.arange(1, n + 1).float().expand(d, n) * (0.75 + torch.rand(d, n, generator=g) / 2),
         "B": _normal(g, tokens, groups, n, dtype=dtype), "C": _normal(g, tokens, groups, n, dtype=dtype),
         "skip": 0.5 + torch.rand(d, generator=g), "gate": _normal(g, tokens, d, dtype=dtype),
         "dt_bias": torch.log(torch.expm1(0.001 * 100 ** torch.rand(d, generator=g))), "softplus": True,
         "slots": torch.tensor(more["slots"], dtype=torch.int32) if "slots" in more else None,
         "state": _normal(g, len(lengths) + 2, d, n) if more.get("state", True) else None}
    if more.get("plain"):
        c.update(skip=None, gate=None, dt_bias=None, softplus=False, dt=c["dt"].abs() * 0.1)
    return c


def _scan_args(c, lengths, packed, more):
    d = c["u"].shape[1]
    lead = () if packed else (len(lengths), lengths[0])

    def rows(t):
        if t is None:
            return None
        shape = t.shape[1:]
        flat = t.reshape(*(lead or t.shape[:1]), -1)
        return _wide(flat, more.get("wide", 0), more.get("shift", 0)).unflatten(-1, tuple(shape))

    args = [rows(c["u"]), rows(c["dt"]), _on(c["A"]).contiguous(), rows(c["B"]), rows(c["C"])]
    kw = {"skip": _on(c["skip"]), "gate": rows(c["gate"]), "dt_bias": _on(c["dt_bias"]), "softplus": c["softplus"],
          "slots": _on(c["slots"])}
    if packed:
        kw["seq_offsets"] = _offsets(lengths)
    return d, args, kw


def _reference(c, lengths, fresh=False, slots=None):
    return ref.scan(c["u"], c["dt"], c["A"], c["B"], c["C"], c["skip"], c["gate"], c["dt_bias"], c["softplus"], c["state"],
                    c["slots"] if slots is None else slots, lengths, fresh)


@pytest.mark.parametrize("i", range(len(SCAN)))
def test_scan_prompt(i):
    kind, lengths, packed, d, n, groups, more = SCAN[i]
    c = _scan_case(i, kind, lengths, d, n, groups, more)
    fresh = more.get("fresh", False)
    want, bound, state, state_bound = _reference(c, lengths, fresh)
    d, args, kw = _scan_args(c, lengths, packed, more)
    for longest in (None, max(lengths)):
        dev_state = _on(c["state"])
        if fresh:
            dev_state[:len(lengths)] = float("nan")
        got = c2d.selective_scan(*args, **kw, state=dev_state, fresh=fresh, longest=longest)
        assert got.shape == args[0].shape
        ref.close(got.reshape(-1, d), want, bound, f"scan {SCAN[i]}")
        if dev_state is not None:
            ref.close(dev_state, state, state_bound, "state")


def test_scan_of_many_short_sequences():
    """More sequences than are put in order of their lengths."""
    g = _rng(40)
    lengths = torch.randint(0, 9, (300,), generator=g).tolist()
    c = _scan_case(41, "f32", lengths, 64, 8, 2, {})
    want, bound, state, state_bound = _reference(c, lengths)
    _, args, kw = _scan_args(c, lengths, True, {})
    dev_state = _on(c["state"])
    ref.close(c2d.selective_scan(*args, **kw, state=dev_state), want, bound, "many")
    ref.close(dev_state, state, state_bound, "state")


def test_scan_token_of_a_large_batch():
    """Past the size where a workgroup takes two sequences, an odd number of them."""
    rows, d, n = 513, 512, 16
    c = _scan_case(42, "bf16", [1] * rows, d, n, 1, {})
    c["slots"] = torch.randperm(rows + 2, generator=_rng(3))[:rows].to(torch.int32)
    c["slots"][5] = -1
    want, bound, state, state_bound = _reference(c, [1] * rows)
    _, args, kw = _scan_args(c, [1] * rows, True, {})
    del kw["seq_offsets"]
    dev_state = _on(c["state"])
    ref.close(c2d.selective_scan_step(*args, **kw, state=dev_state), want, bound, "large batch")
    ref.close(dev_state, state, state_bound, "state")


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,d,n,groups", [(1, 1, 1, 1), (1, 2048, 16, 1), (7, 96, 64, 8), (5, 70, 5, 2), (3, 33, 256, 1),
                                             (2, 260, 130, 1)])
def test_scan_token(kind, rows, d, n, groups):
    c = _scan_case(rows + d, kind, [1] * rows, d, n, groups, {})
    slots = torch.randperm(rows + 2, generator=_rng(2))[:rows].to(torch.int32)
    if rows > 4:
        slots[2], slots[3] = -1, rows + 2
    c["slots"] = slots
    want, bound, state, state_bound = _reference(c, [1] * rows)
    _, args, kw = _scan_args(c, [1] * rows, True, {"wide": 4})
    del kw["seq_offsets"]
    dev_state = _on(c["state"])
    got = c2d.selective_scan_step(*args, **kw, state=dev_state)
    ref.close(got, want, bound, "scan token")
    ref.close(dev_state, state, state_bound, "state")


@pytest.mark.parametrize("split", [1, 16, 700])
def test_prompt_in_two_calls_and_tokens_agree_with_one_call(split):
    """A prompt in two pieces, the first ones' states carried, and its end token by token."""
    lengths, d, n = [900], 64, 16
    c = _scan_case(5, "f32", lengths, d, n, 1, {})
    want, bound, state, state_bound = _reference(c, lengths)
    _, args, kw = _scan_args(c, lengths, False, {})
    kw.pop("gate")
    gate = _on(c["gate"]).reshape(1, -1, d)
    dev_state = _on(c["state"])
    cut = lambda t, a, b: t[:, a:b]  # noqa: E731
    got = []
    for a, b in ((0, split), (split, 880)):
        got.append(c2d.selective_scan(*[t if t.dim() == 2 else cut(t, a, b) for t in args], gate=cut(gate, a, b),
                                      state=dev_state, **kw))
    for t in range(880, 900):
        y = c2d.selective_scan_step(*[v if v.dim() == 2 else v[:, t] for v in args], gate=gate[:, t], state=dev_state, **kw)
        got.append(y[:, None])
    ref.close(torch.cat(got, 1).reshape(-1, d), want, bound, "pieces")
    ref.close(dev_state, state, state_bound, "state")


def test_extreme_steps_and_gates():
    """Step sizes from nothing to where the decay underflows, gates far out; NaN and infinities stay in their channel
    and sequence."""
    lengths, d, n = [40, 40], 64, 16
    c = _scan_case(11, "f32", lengths, d, n, 1, {})
    c["dt"][:, 0] = -200.0  # softplus underflows to 0: the state stays
    c["dt"][:, 1] = 80.0
    c["dt"][:, 2] = -20.0
    c["gate"][:, 3] = -120.0
    c["gate"][:, 4] = 120.0
    want, bound, state, state_bound = _reference(c, lengths)
    _, args, kw = _scan_args(c, lengths, True, {})
    dev_state = _on(c["state"])
    got = c2d.selective_scan(*args, **kw, state=dev_state)
    ref.close(got, want, bound, "extremes")
    ref.close(dev_state, state, state_bound, "state")
    args[0][45, 7] = float("nan")
    args[0][50, 9] = float("inf")
    again_state = _on(c["state"])
    again = c2d.selective_scan(*args, **kw, state=again_state)
    touched = torch.zeros_like(again, dtype=torch.bool)
    touched[45:, 7] = True
    touched[50:, 9] = True
    assert torch.equal(again[~touched], got[~touched])
    assert not torch.isfinite(again[45:, 7]).any() and not torch.isfinite(again[50:, 9]).any()
    keep = torch.ones_like(again_state, dtype=torch.bool)
    keep[1, 7] = keep[1, 9] = False
    assert torch.equal(again_state[keep], dev_state[keep])


# ---------------------------------------------------------------- 4-bit products

W4 = [  # type, rows, in, out, group, zeros, act, residual, before, what else
    ("bf16", 1, 128, 16, 128, False, "none", False, False, {}),
    ("f16", 1, 1, 1, 32, True, "none", False, False, {}),
    ("bf16", 1, 2048, 512, 128, False, "silu", True, False, {}),
    ("f16", 3, 401, 77, 32, True, "relu", True, True, {}),
    ("bf16", 16, 640, 100, 64, True, "none", True, False, {"wide": 8}),
    ("f16", 17, 500, 48, 64, False, "prelu", True, False, {"wide": 3, "shift": 1}),
    ("bf16", 33, 130, 200, 128, True, "none", False, False, {}),
    ("f16", 64, 1024, 64, 32, False, "none", True, True, {"bias": False}),
    ("bf16", 70, 72, 31, 32, False, "silu", False, False, {}),
    ("f16", 8, 4100, 1030, 128, True, "none", False, False, {}),
    ("bf16", 2, 8192, 48, 32, True, "none", False, False, {}),
    # the other shapes of a workgroup: by outputs, rows and inputs
    ("bf16", 12, 1500, 333, 64, True, "none", True, False, {}),
    ("f16", 3, 300, 8200, 128, False, "none", True, False, {}),
    ("bf16", 11, 2090, 8200, 32, True, "relu", False, False, {}),
    ("f16", 16, 777, 16400, 64, True, "none", False, False, {}),
    ("bf16", 9, 1160, 32790, 128, True, "none", True, True, {}),
]


def _w4_case(seed, kind, rows, k, n, group, zeros, act, residual, more):
    g = _rng(seed)
    dtype = TYPES[kind]
    groups = -(-k // group)
    return {"x": _normal(g, rows, k, dtype=dtype),
            "codes": torch.randint(0, 256, (n, (k + 1) // 2), generator=g, dtype=torch.uint8),
            "scales": ((torch.rand(n, groups, generator=g) + 0.5) / (4.6 * k ** 0.5)).to(dtype),
            "zeros": torch.randint(0, 16, (n, groups), generator=g, dtype=torch.uint8) if zeros else None,
            "bias": _normal(g, n, scale=0.1) if more.get("bias", True) else None,
            "alpha": torch.rand(n, generator=g) if act == "prelu" else None,
            "residual": _normal(g, rows, n, dtype=dtype) if residual else None}


@pytest.mark.parametrize("i", range(len(W4)))
def test_w4(i):
    kind, rows, k, n, group, zeros, act, residual, before, more = W4[i]
    c = _w4_case(i, kind, rows, k, n, group, zeros, act, residual, more)
    want, bound = ref.w4(c["x"], c["codes"], c["scales"], c["zeros"], group, c["bias"], c["alpha"], c["residual"], act, before)
    weights = c2d.w4_pack(_on(c["codes"]), _on(c["scales"]), _on(c["zeros"]), in_features=k, group=group)
    wide, shift = more.get("wide", 0), more.get("shift", 0)
    x = _wide(c["x"], wide, shift)
    r = None if c["residual"] is None else _wide(c["residual"], wide, shift)
    got = c2d.matvec_w4(x, weights, _on(c["bias"]), _on(c["alpha"]), r, act=act, res_before_act=before)
    ref.close(got, want, bound, f"w4 {W4[i]}")
    out = torch.full((rows, n + 5), float("nan"), dtype=c["x"].dtype, device=DEV)
    c2d.matvec_w4(x, weights, _on(c["bias"]), _on(c["alpha"]), r, act=act, res_before_act=before, out=out[:, :n])
    assert torch.equal(out[:, :n], got) and torch.isnan(out[:, n:]).all()


def test_w4_rows_do_not_mix():
    """A row of x with NaN or an infinity leaves the other rows as they were."""
    c = _w4_case(3, "bf16", 5, 300, 90, 64, True, "none", False, {})
    weights = c2d.w4_pack(_on(c["codes"]), _on(c["scales"]), _on(c["zeros"]), in_features=300, group=64)
    x = _on(c["x"])
    before = c2d.matvec_w4(x, weights)
    x[1, 17] = float("nan")
    x[3, 200] = float("inf")
    after = c2d.matvec_w4(x, weights)
    for r in (0, 2, 4):
        assert torch.equal(before[r], after[r])
    assert torch.isnan(after[1]).all() and not torch.isfinite(after[3]).any()


# ---------------------------------------------------------------- common

def test_empty_calls():
    z = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
    w = torch.ones(8, 4, device=DEV)
    state = torch.ones(3, 3, 8, device=DEV)
    assert c2d.causal_conv1d(z(0, 5, 8), w).shape == (0, 5, 8)
    assert c2d.causal_conv1d(z(2, 0, 8), w, state=state).shape == (2, 0, 8)
    assert (state == 1).all()
    c2d.causal_conv1d(z(2, 0, 8), w, state=state, fresh=True)
    assert (state[:2] == 0).all() and (state[2] == 1).all()
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert c2d.causal_conv1d(z(0, 8), w, seq_offsets=none).shape == (0, 8)
    assert c2d.causal_conv1d_step(z(0, 8), w, state=state).shape == (0, 8)
    A, hs = -torch.ones(8, 4, device=DEV), torch.ones(3, 8, 4, device=DEV)
    assert c2d.selective_scan(z(0, 5, 8), z(0, 5, 8), A, z(0, 5, 1, 4), z(0, 5, 1, 4)).shape == (0, 5, 8)
    empty = torch.zeros(3, dtype=torch.int32, device=DEV)
    c2d.selective_scan(z(0, 8), z(0, 8), A, z(0, 1, 4), z(0, 1, 4), state=hs, seq_offsets=empty)
    assert (hs == 1).all()
    c2d.selective_scan(z(0, 8), z(0, 8), A, z(0, 1, 4), z(0, 1, 4), state=hs, seq_offsets=empty, fresh=True)
    assert (hs[:2] == 0).all() and (hs[2] == 1).all()
    assert c2d.selective_scan_step(z(0, 8), z(0, 8), A, z(0, 1, 4), z(0, 1, 4), state=hs).shape == (0, 8)
    codes = torch.zeros(4, 16, dtype=torch.uint8, device=DEV)
    wt = c2d.w4_pack(codes, torch.ones(4, 1, dtype=torch.bfloat16, device=DEV), group=32)
    assert c2d.matvec_w4(z(0, 32).bfloat16(), wt).shape == (0, 4)


def test_wrong_offsets_touch_no_other_memory():
    """Offsets out of range or out of order are clamped on the device: rows around the tensors stay as they were."""
    d = 64
    x = torch.randn(50, d, device=DEV)
    out = torch.full((150, d), 3.0, device=DEV)
    bad = torch.tensor([-7, 1000, 20, 5, 2000000000], dtype=torch.int32, device=DEV)
    c2d.causal_conv1d(x, torch.randn(d, 4, device=DEV), seq_offsets=bad, out=out[50:100])
    assert (out[:50] == 3).all() and (out[100:] == 3).all()
    b = torch.randn(50, 1, 16, device=DEV)
    c2d.selective_scan(x, x, -torch.ones(d, 16, device=DEV), b, b, softplus=True, seq_offsets=bad, out=out[50:100])
    assert (out[:50] == 3).all() and (out[100:] == 3).all()


def test_long_caches_past_32_bits():
    """State rows and token rows whose offsets pass 2^31 elements."""
    d, n = 1024, 16
    rows = (1 << 31) // (d * n) + 2
    state = torch.empty(rows, d, n, device=DEV)
    c = _scan_case(3, "bf16", [1, 1], d, n, 1, {})
    state[rows - 1] = c["state"][0].to(DEV)
    state[0] = c["state"][1].to(DEV)
    slots = torch.tensor([rows - 1, 0], dtype=torch.int32)
    want, bound, after, after_bound = _reference({**c, "slots": None}, [1, 1])
    _, args, kw = _scan_args(c, [1, 1], True, {})
    kw["slots"] = slots.to(DEV)
    ref.close(c2d.selective_scan(*args, **kw, state=state), want, bound, "far state")
    ref.close(state[[rows - 1, 0]], after[:2], after_bound[:2], "state")
    del state
    tokens, stride = 67, 1 << 25
    far = torch.empty_strided((tokens, 64), (stride, 1), dtype=torch.bfloat16, device=DEV)
    x = torch.randn(tokens, 64, generator=_rng(1)).bfloat16()
    far.copy_(x)
    w = torch.randn(64, 4, device=DEV).bfloat16()
    assert (tokens - 1) * stride > 1 << 31
    assert torch.equal(c2d.causal_conv1d(far[None], w), c2d.causal_conv1d(x.to(DEV)[None], w))
    bc = torch.randn(tokens, 1, 16, device=DEV).bfloat16()
    A = -torch.ones(64, 16, device=DEV)
    near = c2d.selective_scan(x.to(DEV)[None], x.to(DEV)[None], A, bc[None], bc[None], softplus=True)
    assert torch.equal(c2d.selective_scan(far[None], far[None], A, bc[None], bc[None], softplus=True), near)


def test_same_bits_every_time_and_on_another_stream():
    c = _scan_case(21, "bf16", [700, 1, 0, 1300], 128, 16, 1, {})
    _, args, kw = _scan_args(c, [700, 1, 0, 1300], True, {})
    first_state = _on(c["state"])
    first = c2d.selective_scan(*args, **kw, state=first_state)
    w4c = _w4_case(4, "f16", 4, 1000, 500, 64, True, "none", False, {})
    weights = c2d.w4_pack(_on(w4c["codes"]), _on(w4c["scales"]), _on(w4c["zeros"]), in_features=1000, group=64)
    x4 = _on(w4c["x"])
    y4 = c2d.matvec_w4(x4, weights)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, None, side):
        state = _on(c["state"])
        torch.cuda.synchronize()
        y = c2d.selective_scan(*args, **kw, state=state, stream=stream)
        z = c2d.matvec_w4(x4, weights, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(y, first) and torch.equal(state, first_state) and torch.equal(z, y4)


def test_token_calls_in_a_graph():
    """The single-token calls record into a HIP graph; every replay moves the states on as an eager call does."""
    rows, d, n = 3, 128, 16
    g = _rng(8)
    x = _normal(g, rows, d, dtype=torch.bfloat16).to(DEV)
    w = _normal(g, d, 4, dtype=torch.bfloat16).to(DEV)
    conv_state = _normal(g, rows, 3, d, dtype=torch.bfloat16).to(DEV)
    c = _scan_case(9, "bf16", [1] * rows, d, n, 1, {})
    _, args, kw = _scan_args(c, [1] * rows, True, {})
    del kw["seq_offsets"]
    scan_state = _on(c["state"])
    q = _w4_case(1, "bf16", rows, d, d, 32, False, "none", False, {})
    weights = c2d.w4_pack(_on(q["codes"]), _on(q["scales"]), group=32)

    def token(conv_state, scan_state):
        v = c2d.causal_conv1d_step(x, w, state=conv_state, act="silu")
        y = c2d.selective_scan_step(v, *args[1:], **kw, state=scan_state)
        return c2d.matvec_w4(y, weights)

    eager = [s.clone() for s in (conv_state, scan_state)]
    warm = [s.clone() for s in (conv_state, scan_state)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        token(*warm)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token(conv_state, scan_state)
    for _ in range(4):
        want = token(*eager)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert torch.equal(conv_state, eager[0]) and torch.equal(scan_state, eager[1])


def test_binding_refuses():
    """Shapes, types, devices and layouts that the binding names before calling the library."""
    d, n = 8, 4
    x = torch.zeros(2, 5, d, device=DEV)
    w = torch.zeros(d, 4, device=DEV)
    bc = torch.zeros(2, 5, 1, n, device=DEV)
    A = torch.zeros(d, n, device=DEV)
    i32 = torch.zeros(3, dtype=torch.int32, device=DEV)
    state = torch.zeros(2, 3, d, device=DEV)
    hs = torch.zeros(2, d, n, device=DEV)
    wt = c2d.w4_pack(torch.zeros(4, 16, dtype=torch.uint8, device=DEV), torch.ones(4, 1, device=DEV).half(), group=32)
    bad = [lambda: c2d.causal_conv1d(x[0], w), lambda: c2d.causal_conv1d(x, w[:4]), lambda: c2d.causal_conv1d(x, w.half()),
           lambda: c2d.causal_conv1d(x, w.cpu()), lambda: c2d.causal_conv1d(x, w, act="tanh"),
           lambda: c2d.causal_conv1d(x, w, torch.zeros(d, device=DEV).half()),
           lambda: c2d.causal_conv1d(x, w, torch.zeros(d - 1, device=DEV)),
           lambda: c2d.causal_conv1d(x.transpose(1, 2), torch.zeros(5, 4, device=DEV)),
           lambda: c2d.causal_conv1d(x, w, state=state[:, :2]), lambda: c2d.causal_conv1d(x, w, state=state.half()),
           lambda: c2d.causal_conv1d(x, w, state=state, slots=i32), lambda: c2d.causal_conv1d(x, w, slots=i32[:2].long()),
           lambda: c2d.causal_conv1d(x[0], w, seq_offsets=i32.long()), lambda: c2d.causal_conv1d(x, w, seq_offsets=i32),
           lambda: c2d.causal_conv1d(x, w, out=torch.empty(2, 5, d + 1, device=DEV)),
           lambda: c2d.causal_conv1d_step(x, w, state=state),
           lambda: c2d.selective_scan(x, x[:, :4], A, bc, bc), lambda: c2d.selective_scan(x, x, A[:4], bc, bc),
           lambda: c2d.selective_scan(x, x, A, bc[:, :, 0], bc), lambda: c2d.selective_scan(x, x, A, bc, bc[..., :2]),
           lambda: c2d.selective_scan(x, x, A.half(), bc, bc), lambda: c2d.selective_scan(x, x, A, bc, bc, gate=x.half()),
           lambda: c2d.selective_scan(x, x, A, bc, bc, state=hs.half()),
           lambda: c2d.selective_scan(x, x, A, bc, bc, state=hs[..., :2]),
           lambda: c2d.selective_scan(x, x, A, bc, bc, skip=torch.zeros(3, device=DEV)),
           lambda: c2d.selective_scan_step(x, x, A, bc, bc, state=hs),
           lambda: c2d.matvec_w4(torch.zeros(1, 32, device=DEV), wt), lambda: c2d.matvec_w4(torch.zeros(32, device=DEV).half(), wt),
           lambda: c2d.matvec_w4(torch.zeros(1, 31, device=DEV).half(), wt),
           lambda: c2d.w4_pack(torch.zeros(4, 16, device=DEV), torch.ones(4, 1, device=DEV).half(), group=32),
           lambda: c2d.w4_pack(torch.zeros(4, 16, dtype=torch.uint8, device=DEV), torch.ones(4, 2, device=DEV).half(), group=32)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", i)
    library = [lambda: c2d.causal_conv1d(x, torch.zeros(d, 5, device=DEV)), lambda: c2d.causal_conv1d(x, w, act="prelu"),
               lambda: c2d.causal_conv1d(x, w, out=x), lambda: c2d.causal_conv1d(x, w, out=x[:, :1].expand(2, 5, d)),
               lambda: c2d.selective_scan(x, x, A, bc.expand(2, 5, 3, n).contiguous(), bc.expand(2, 5, 3, n).contiguous()),
               lambda: c2d.selective_scan(x, x, A, bc, bc, out=x),
               lambda: c2d.w4_pack(torch.zeros(4, 16, dtype=torch.uint8, device=DEV), torch.ones(4, 1, device=DEV).half(), group=48)]
    for call in library:
        with pytest.raises(c2d.Conv2dError) as e:
            call()
        assert e.value.code == c2d.EINVAL


def _long_scan(lengths, d=64, n=16, packed=True, kind="f32", groups=1):
    c = _scan_case(31, kind, lengths, d, n, groups, {})
    return c, _scan_args(c, lengths, packed, {})


def _workspace_of(args, kw, lengths, packed, **more):
    """What the library wants for a call, from the struct that the binding would pass."""
    import ctypes
    from conv2d_bias_activation_amd import sequence
    taken = []
    real = sequence._call
    sequence._call = lambda name, packed_args, device, stream: taken.append(packed_args)
    try:
        c2d.selective_scan(*args, **kw, workspace=False, **more)
    finally:
        sequence._call = real
    size = ctypes.c_size_t(0)
    assert c2d._load().selective_scan_workspace_size(taken[0], ctypes.byref(size)) == c2d.OK
    return size.value


@pytest.mark.parametrize("lengths,packed,n,groups", [([3000], False, 16, 1), ([2000, 1, 0, 900, 64, 65], True, 16, 1),
                                                     ([1500, 1500], False, 64, 2), ([1024, 1023, 1025], True, 5, 1),
                                                     ([1300], True, 130, 1)])
def test_split_scans(lengths, packed, n, groups):
    """Sequences cut into chunks that run side by side: the right values with the workspace, without it, and the same
    bits again; a workspace one byte short is not written."""
    c, (d, args, kw) = _long_scan(lengths, n=n, packed=packed, groups=groups)
    want, bound, state, state_bound = _reference(c, lengths)
    need = _workspace_of(args, kw, lengths, packed, longest=max(lengths))
    assert need > 0
    seen = []
    for ws in (None, False, torch.empty(need, dtype=torch.uint8, device=DEV), None):
        dev_state = _on(c["state"])
        y = c2d.selective_scan(*args, **kw, state=dev_state, longest=max(lengths), workspace=ws)
        ref.close(y.reshape(-1, d), want, bound, f"split {lengths}")
        ref.close(dev_state, state, state_bound, "state")
        seen.append((y, dev_state))
    for y, s in seen[2:]:
        assert torch.equal(y, seen[0][0]) and torch.equal(s, seen[0][1])
    short = torch.full((need,), 77, dtype=torch.uint8, device=DEV)[:need - 1]
    dev_state = _on(c["state"])
    y = c2d.selective_scan(*args, **kw, state=dev_state, longest=max(lengths), workspace=short)
    assert (short == 77).all() and torch.equal(y, seen[1][0]) and torch.equal(dev_state, seen[1][1])


def test_split_scan_of_wrong_offsets_stays_in_its_workspace():
    d, n = 64, 16
    x = torch.randn(4000, d, device=DEV)
    b = torch.randn(4000, 1, n, device=DEV)
    bad = torch.tensor([900, -5, 4000, 17, 3999, 2000000000], dtype=torch.int32, device=DEV)
    args, kw = (x, x, -torch.ones(d, n, device=DEV), b, b), {"softplus": True, "seq_offsets": bad}
    need = _workspace_of(args, kw, None, True, longest=4000)
    assert need > 0
    room = torch.full((need + 512,), 77, dtype=torch.uint8, device=DEV)
    out = torch.full((4200, d), 3.0, device=DEV)
    c2d.selective_scan(*args, **kw, longest=4000, workspace=room[256:256 + need], out=out[100:4100])
    assert (room[:256] == 77).all() and (room[256 + need:] == 77).all()
    assert (out[:100] == 3).all() and (out[4100:] == 3).all()
