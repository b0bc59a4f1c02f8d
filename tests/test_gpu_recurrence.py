"""The gated linear recurrence, its single-token form and its gradient on the GPU against their definitions in 64 bits."""
import pytest
import torch

import recurrence_reference as rec
import sequence_reference as ref

pytestmark = pytest.mark.gpu

c2d = pytest.importorskip("conv2d_bias_activation_amd")
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

CASES = [  # type, lengths, packed, channels, what else
    ("f32", [1], False, 1, {}),
    ("bf16", [77], False, 512, {}),
    ("f16", [16, 16], False, 64, {"slots": [2, 0]}),
    ("bf16", [63], False, 126, {"coupled": False}),
    ("bf16", [64, 64, 64], False, 72, {"wide": 8}),
    ("f16", [65], False, 40, {"wide": 3, "shift": 1}),
    ("f32", [130, 0, 1, 2, 3, 7, 8, 9, 63, 64, 65], True, 36, {"slots": [10, 3, 1, 0, 5, 4, 2, 6, 7, 8, 9]}),
    ("bf16", [0, 0, 31, 1, 0, 48, 2], True, 1032, {"slots": [0, 1, 2, 3, 4, 5, 6], "wide": 1032}),
    ("f16", [7, 64, 9], True, 13, {"slots": [1, -1, 5]}),
    ("bf16", [3, 20], True, 264, {"state": False}),
    ("f32", [1, 0, 140], True, 129, {"bias": False, "fresh": True}),
    ("bf16", [2, 0, 300], True, 128, {"fresh": True, "wide": 64, "gate": False}),
    ("bf16", [700, 3, 1201, 0], True, 96, {"slots": [3, 2, 1, 0]}),
    ("f16", [1500], False, 103, {"coupled": False, "gate": False}),
    ("f32", [900, 900], False, 70, {"slots": [-1, 0]}),
    ("f32", [600, 1, 129], True, 33, {"coupled": False, "state": False}),
    ("bf16", [2049], False, 130, {"longest": 2049}),
    # several rounds of workgroups, of equal sequences in chunks
    ("f32", [900, 900, 900], False, 2056, {}),
    ("bf16", [1100, 1100], False, 3330, {"coupled": False}),
    # many sequences whose rows share cache lines between blocks of channels; the second lot taken by length, too
    ("bf16", [(i * 29) % 83 for i in range(70)], True, 1001, {"longest": 82}),
    ("f16", [(i * 53) % 257 + 9 * (i % 3) for i in range(64)], True, 701, {"longest": 274, "slots": list(range(63, -1, -1))}),
    # many whole sequences, taken by length
    ("bf16", [(i * 37) % 101 for i in range(20)], True, 4101, {"slots": list(range(19, -1, -1)), "longest": 100}),
    ("f32", [3, 90, 0, 0, 90, 17, 90, 1, 64, 65, 2, 120, 119, 5, 77, 0, 31, 90], True, 2020, {"longest": 120}),
]


def _case(seed, kind, lengths, packed, d, more):
    g = torch.Generator().manual_seed(seed)
    dtype, n = TYPES[kind], sum(lengths)
    r = lambda *s, scale=1.0, dtype=dtype: (torch.randn(*s, generator=g) * scale).to(dtype)
    c = {"x": r(n, d), "forget": r(n, d), "gate": r(n, d) if more.get("gate", True) else None,
         "bias": torch.rand(d, generator=g) * 6 - 0.5 if more.get("bias", True) else None,
         "coupled": more.get("coupled", True), "slots": more.get("slots"),
         "state": r(len(lengths) + 2, d, dtype=torch.float32) if more.get("state", True) else None,
         "grad": r(n, d), "grad_state": r(len(lengths) + 2, d, dtype=torch.float32) if more.get("state", True) else None}
    return c


def _on(t):
    return None if t is None else (torch.tensor(t, dtype=torch.int32) if isinstance(t, list) else t).to(DEV)


def _offsets(lengths):
    return torch.tensor([0] + lengths).cumsum(0).to(torch.int32).to(DEV)


def _rows(t, lengths, packed, more):
    """The token rows on the GPU as columns of a wider tensor whose other columns are NaN."""
    if t is None:
        return None
    t = t if packed else t.reshape(len(lengths), lengths[0], -1)
    shift, extra = more.get("shift", 0), more.get("wide", 0)
    wide = torch.full((*t.shape[:-1], t.shape[-1] + extra + shift), float("nan"), dtype=t.dtype, device=DEV)
    view = wide[..., shift:shift + t.shape[-1]]
    view.copy_(t)
    return view


def _kw(c, lengths, packed, more):
    kw = {"gate": _rows(c["gate"], lengths, packed, more), "forget_bias": _on(c["bias"]), "coupled": c["coupled"],
          "slots": _on(c["slots"])}
    if packed:
        kw.update(seq_offsets=_offsets(lengths), longest=more.get("longest"))
    return kw


@pytest.mark.parametrize("workspace", [None, False])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_prompt(i, workspace):
    kind, lengths, packed, d, more = CASES[i]
    c = _case(i, *CASES[i])
    fresh = more.get("fresh", False)
    want, bound, new, new_bound, _ = rec.forward(c["x"], c["forget"], c["gate"], c["bias"], c["coupled"], c["state"],
                                                 c["slots"], lengths, fresh)
    state = _on(c["state"])
    if fresh and state is not None:
        state[:len(lengths)] = float("nan")  # it may hold anything
    x = _rows(c["x"], lengths, packed, more)
    got = c2d.gated_recurrence(x, _rows(c["forget"], lengths, packed, more), state=state, fresh=fresh, workspace=workspace,
                               **_kw(c, lengths, packed, more))
    assert got.shape == x.shape
    ref.close(got.reshape(-1, d), want, bound, f"{CASES[i]}")
    if state is not None:
        ref.close(state, new, new_bound, f"state {CASES[i]}")


@pytest.mark.parametrize("i", range(len(CASES)))
def test_gradient(i):
    kind, lengths, packed, d, more = CASES[i]
    c = _case(i + 100, *CASES[i])
    start = None if more.get("fresh") else c["state"]
    want = rec.backward(c["grad"], c["x"], c["forget"], c["gate"], c["bias"], c["coupled"], start, c["grad_state"], c["slots"],
                        lengths)
    r = lambda name: _rows(c[name], lengths, packed, more)
    state, grad_state = _on(start), _on(c["grad_state"])
    got = c2d.gated_recurrence_backward(r("grad"), r("x"), r("forget"), state=state, grad_state=grad_state,
                                        **_kw(c, lengths, packed, more))
    for name, g, (value, bound) in zip(["x", "forget", "gate", "bias", "state"], [*got, grad_state], want):
        if name == "bias" and c["bias"] is None or value is None:
            assert g is None
            continue
        ref.close(g.reshape(value.shape), value, bound, f"{name} of {CASES[i]}")
    if start is not None:
        assert torch.equal(state.cpu(), start)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,d,more", [(1, 1, {}), (1, 2048, {}), (9, 264, {"coupled": False}), (5, 77, {"wide": 1}),
                                         (3, 40, {"gate": False, "bias": False}), (6, 72, {"shift": 4, "wide": 4})])
def test_token(kind, rows, d, more):
    c = _case(rows + d, kind, [1] * rows, True, d, more)
    slots = torch.randperm(rows + 2, generator=torch.Generator().manual_seed(1))[:rows].tolist()
    if rows > 4:
        slots[2], slots[3] = -1, rows + 2  # rows without a state
    want, bound, new, new_bound, _ = rec.forward(c["x"], c["forget"], c["gate"], c["bias"], c["coupled"], c["state"], slots,
                                                 [1] * rows)
    state = _on(c["state"])
    r = lambda name: _rows(c[name], [1] * rows, True, more)
    got = c2d.gated_recurrence_step(r("x"), r("forget"), state=state, gate=r("gate"), forget_bias=_on(c["bias"]),
                                    coupled=c["coupled"], slots=_on(slots))
    ref.close(got, want, bound, "token")
    ref.close(state, new, new_bound, "token state")


def test_tokens_continue_a_prompt():
    """A prompt, then tokens one by one, ends as the whole prompt does, to the rounding of either."""
    d, n = 96, 200
    g = torch.Generator().manual_seed(4)
    x, z = torch.randn(1, n, d, generator=g), torch.randn(1, n, d, generator=g)
    want, bound, new, new_bound, _ = rec.forward(x[0], z[0], None, None, True, torch.zeros(1, d), None, [n])
    state = torch.zeros(1, d, device=DEV)
    x, z = x.to(DEV), z.to(DEV)
    ys = [c2d.gated_recurrence(x[:, :190], z[:, :190], state=state)[0]]
    for t in range(190, n):
        ys.append(c2d.gated_recurrence_step(x[:, t], z[:, t], state=state))
    ref.close(torch.cat(ys), want, bound, "prompt and tokens")
    ref.close(state, new, new_bound, "their state")


def test_many_chunks_are_the_unsplit_call():
    """A document split over many chunks against the call without a workspace, which walks it in one."""
    n, d = 40000, 64
    g = torch.Generator(device=DEV).manual_seed(5)
    x, z = (torch.randn(1, n, d, generator=g, device=DEV) for _ in range(2))
    bias = torch.rand(d, generator=g, device=DEV) * 6
    a, b = (torch.randn(1, d, generator=g, device=DEV) for _ in range(2))
    b.copy_(a)
    y = c2d.gated_recurrence(x, z, forget_bias=bias, state=a)
    w = c2d.gated_recurrence(x, z, forget_bias=bias, state=b, workspace=False)
    # either is off by some gates' roundings (twelve of 2^-24 a token) over a memory of under 500 tokens
    size = 5.0  # |h| stays under the largest |x|
    assert (y - w).abs().max() <= 2 * 500 * 12 * ref.U32 * size
    assert (a - b).abs().max() <= 2 * 500 * 12 * ref.U32 * size


def test_gradients_as_slices_of_one_tensor():
    c = _case(7, "bf16", [50, 21], True, 64, {})
    kw = _kw(c, [50, 21], True, {})
    args = [_on(c[k]) for k in ("grad", "x", "forget")]
    want = c2d.gated_recurrence_backward(*args, **kw)
    whole = torch.full((71, 192), float("nan"), dtype=torch.bfloat16, device=DEV)
    out = whole[:, 64:128], whole[:, :64], whole[:, 128:]
    got = c2d.gated_recurrence_backward(*args, out=out, **kw)
    assert got[0] is out[0]
    for g, w in zip(got, want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("lengths,rows,d", [([30, 0, 41], 100, 40), ([500, 1, 300], 900, 130)])
def test_rows_behind_the_last_sequence_stay(lengths, rows, d):
    """A padded packed batch: rows that no sequence covers are neither read into a result nor written."""
    n = sum(lengths)
    c = _case(n, "bf16", [rows], True, d, {"state": False})
    kw = _kw(c, lengths, True, {})
    args = [_on(c[k]) for k in ("grad", "x", "forget")]
    for t in (*args, kw["gate"]):
        t[n:] = float("nan")
    cut = {**kw, "gate": kw["gate"][:n]}
    outs = [torch.full((rows, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    c2d.gated_recurrence(args[1], args[2], out=outs[3], **kw)
    got = c2d.gated_recurrence_backward(*args, out=tuple(outs[:3]), **kw)
    want_y = c2d.gated_recurrence(args[1][:n], args[2][:n], workspace=False, **cut)
    want = c2d.gated_recurrence_backward(*(t[:n] for t in args), **cut)
    # the two calls may be cut differently, so they are compared with the definition
    for o in outs:
        assert (o[n:] == 7).all()
    y, bound, *_ = rec.forward(c["x"][:n], c["forget"][:n], c["gate"][:n], c["bias"], True, None, None, lengths)
    ref.close(outs[3][:n], y, bound, "padded")
    ref.close(want_y, y, bound, "not padded")
    grads = rec.backward(c["grad"][:n], c["x"][:n], c["forget"][:n], c["gate"][:n], c["bias"], True, None, None, None, lengths)
    for g, w, (value, bound) in zip(got, want, grads):
        ref.close(g[:n] if g.dim() == 2 else g, value, bound, "padded gradient")
        ref.close(w, value, bound, "gradient")


def test_offsets_past_32_bits():
    """Rows so far apart that an element's index passes 2^31, read and written in place."""
    d, n, pitch = 8, 300, 1 << 23
    whole = torch.empty(n * pitch + 64, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(8)
    view = lambda first: whole[first:first + n * pitch].view(n, pitch)[:, :d]
    x, z = torch.randn(n, d, generator=g, device=DEV).bfloat16(), torch.randn(n, d, generator=g, device=DEV).bfloat16()
    view(0).copy_(x)
    view(16).copy_(z)
    offsets = _offsets([100, 200])
    y = c2d.gated_recurrence(view(0), view(16), seq_offsets=offsets)
    assert torch.equal(y, c2d.gated_recurrence(x, z, seq_offsets=offsets))
    got = c2d.gated_recurrence_backward(y, view(0), view(16), seq_offsets=offsets)
    for a, b in zip(got, c2d.gated_recurrence_backward(y, x, z, seq_offsets=offsets)):
        assert (a is None and b is None) or torch.equal(a, b)


def test_infinities_stay_in_their_channel_and_sequence():
    lengths, d = [70, 5, 600], 40
    c = _case(9, "f32", lengths, True, d, {})
    bad = {"x": (10, 3, float("inf")), "forget": (80, 7, float("nan")), "gate": (300, 11, float("-inf"))}
    poisoned = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    for name, (t, ch, v) in bad.items():
        poisoned[name][t, ch] = v
    off = torch.ones(sum(lengths), d, dtype=torch.bool)
    off[10:70, 3] = False
    off[75:, 7] = False
    off[300, 11] = False

    def run(c):
        state = _on(c["state"])
        kw = _kw(c, lengths, True, {})
        y = c2d.gated_recurrence(_on(c["x"]), _on(c["forget"]), state=state, **kw)
        grads = c2d.gated_recurrence_backward(_on(c["grad"]), _on(c["x"]), _on(c["forget"]), state=_on(c["state"]), **kw)
        return y.cpu(), [g.cpu() for g in grads], state.cpu()

    y, grads, state = run(c)
    py, pgrads, pstate = run(poisoned)
    assert torch.equal(y[off], py[off])
    clean = torch.ones(d, dtype=torch.bool)
    clean[[3, 7, 11]] = False
    for a, b in zip(grads, pgrads):
        assert torch.equal(a[..., clean], b[..., clean])
    assert torch.equal(grads[0][75:, 3], pgrads[0][75:, 3])  # the same channel of the other sequences
    assert torch.equal(state[:, clean], pstate[:, clean])


def test_gates_at_their_ends():
    """Forget gates that are shut or open to the last bit: the state is taken over or kept, exactly."""
    d = 16
    x = torch.randn(1, 100, d, generator=torch.Generator().manual_seed(3)).to(DEV)
    state = torch.full((1, d), 1e30, device=DEV)
    y = c2d.gated_recurrence(x, torch.full_like(x, float("-inf")), state=state)
    assert torch.equal(y, x) and torch.equal(state, x[:, -1])
    state = torch.full((1, d), 3.0, device=DEV)
    y = c2d.gated_recurrence(x, torch.full_like(x, float("inf")), state=state)
    assert (y == 3).all() and (state == 3).all()
    y = c2d.gated_recurrence(x, torch.full_like(x, 3e38), forget_bias=torch.full((d,), 3e38, device=DEV), state=state)
    assert (y == 3).all()


def test_captured_calls_replay():
    lengths, d = [400, 0, 90], 64
    c = _case(12, "bf16", lengths, True, d, {})
    kw = _kw(c, lengths, True, {})
    x, z, e = _on(c["x"]), _on(c["forget"]), _on(c["grad"])
    start, gs0 = _on(c["state"]), _on(c["grad_state"])
    state, gs = start.clone(), gs0.clone()
    want_y = c2d.gated_recurrence(x, z, state=state, **kw)
    want = c2d.gated_recurrence_backward(e, x, z, state=start, grad_state=gs, **kw)
    s2, gs2 = start.clone(), gs0.clone()
    ws = torch.empty(8 << 20, dtype=torch.uint8, device=DEV)
    ws2 = torch.empty(8 << 20, dtype=torch.uint8, device=DEV)
    outs = tuple(torch.empty_like(x) for _ in range(3))
    y = torch.empty_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c2d.gated_recurrence(x, z, state=s2, out=y, workspace=ws, **kw)
        got = c2d.gated_recurrence_backward(e, x, z, state=start, grad_state=gs2, out=outs, workspace=ws2, **kw)
    for _ in range(3):
        s2.copy_(start)
        gs2.copy_(gs0)
        y.zero_()
        ws.fill_(255)
        ws2.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(s2, state) and torch.equal(gs2, gs)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_calls_on_other_streams():
    d = 128
    g = torch.Generator(device=DEV).manual_seed(2)
    x, z, e = (torch.randn(3, 700, d, generator=g, device=DEV).bfloat16() for _ in range(3))
    want = c2d.gated_recurrence(x, z), c2d.gated_recurrence_backward(e, x, z)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [(c2d.gated_recurrence(x, z, stream=s), c2d.gated_recurrence_backward(e, x, z, stream=s)) for s in streams]
    torch.cuda.synchronize()
    for y, grads in got:
        assert torch.equal(y, want[0])
        for a, b in zip(grads[:2], want[1][:2]):
            assert torch.equal(a, b)


def test_gradient_needs_a_workspace():
    x = torch.zeros(1, 10, 8, device=DEV)
    with pytest.raises(c2d.Conv2dError, match="needs a workspace"):
        c2d.gated_recurrence_backward(x, x, x, workspace=False)


def test_nothing_to_do():
    e = torch.zeros(0, 8, device=DEV)
    bias = torch.ones(8, device=DEV)
    offsets = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert c2d.gated_recurrence(e, e, seq_offsets=offsets).shape == (0, 8)
    got = c2d.gated_recurrence_backward(e, e, e, forget_bias=bias, seq_offsets=offsets)
    assert torch.equal(got[3], torch.zeros(8, device=DEV))
    state = torch.ones(3, 8, device=DEV)
    offsets = torch.zeros(4, dtype=torch.int32, device=DEV)
    c2d.gated_recurrence(e, e, state=state, seq_offsets=offsets)
    assert (state == 1).all()
    got = c2d.gated_recurrence_backward(e, e, e, forget_bias=bias, grad_state=state, seq_offsets=offsets)
    assert (got[3] == 0).all() and (state == 1).all()
    c2d.gated_recurrence(e, e, state=state, seq_offsets=offsets, fresh=True)
    assert (state == 0).all()
    assert c2d.gated_recurrence_step(e, e, state=state).shape == (0, 8)
