"""Cases of the gated linear recurrence, for prompts, single tokens and gradients, and of products in 8-bit integers.

``run`` computes a case with the library's operators where ``own`` is true, and otherwise in plain 32-bit torch
operations. ``exact`` computes the definition in 64 bits, one token at a time.

The sizes are those of a recurrent block of 240 to 4096 channels: a projection makes the 3*D columns "x | forget | gate"
that the recurrence reads as slices, sequences of a batch have different lengths (empty ones and single tokens among
them), states live in a pool whose rows the sequences name, and the projections multiply 16-bit tokens, quantized as they
come, with 8-bit weights.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # a short prompt of one user, on a narrow block: latency
        {"name": "recurrence prompt short", "op": "rec", "type": "f16", "seqs": 1, "tokens": 77, "channels": 512, "packed": False},
        # one long document: few channels, many tokens
        {"name": "recurrence prompt long", "op": "rec", "type": "bf16", "seqs": 1, "tokens": 65536, "channels": 1024, "packed": False},
        # a prefill batch of ragged prompts, packed, on a wide block
        {"name": "recurrence prompt batch", "op": "rec", "type": "bf16", "seqs": 16, "tokens": 32768, "channels": 4096, "packed": True},
        # one user's next token
        {"name": "recurrence token one", "op": "rec_step", "type": "bf16", "seqs": 1, "channels": 2048},
        # a full decode batch
        {"name": "recurrence token batch", "op": "rec_step", "type": "f16", "seqs": 512, "channels": 4096},
        # training in 32 bits on a few short packed texts, odd sizes
        {"name": "recurrence gradient odd", "op": "rec_grad", "type": "f32", "seqs": 3, "tokens": 999, "channels": 250, "packed": True},
        # training on one long document in 16 bits
        {"name": "recurrence gradient long", "op": "rec_grad", "type": "f16", "seqs": 1, "tokens": 32768, "channels": 1024, "packed": False},
        # a training batch
        {"name": "recurrence gradient batch", "op": "rec_grad", "type": "bf16", "seqs": 8, "tokens": 32768, "channels": 2048, "packed": False},
        # a projection of one user's token
        {"name": "product one row", "op": "q8", "type": "bf16", "rows": 1, "in": 2048, "out": 4096, "pair": False},
        # a decode batch, odd sizes: rows, inputs and outputs end inside a tile
        {"name": "product decode odd", "op": "q8", "type": "f16", "rows": 37, "in": 4010, "out": 10007, "pair": False},
        # a short prompt through two projections that share its quantized rows
        {"name": "product pair", "op": "q8", "type": "bf16", "rows": 333, "in": 2048, "out": 4096, "pair": True},
        # a prefill batch through a wide projection
        {"name": "product prompt", "op": "q8", "type": "bf16", "rows": 4096, "in": 4096, "out": 16384, "pair": False},
    ]


def _spread(rng, low, high):
    """A whole number between the two, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _channels(rng, low, high):
    """Channel counts: powers of two, odd multiples of 64 and of 8, or any number."""
    n = _spread(rng, low, high)
    kind = rng.randrange(4)
    if kind == 0:
        return 1 << min(max(round(math.log2(n)), math.ceil(math.log2(low))), int(math.log2(high)))
    if kind == 3:
        return n
    step = 64 if kind == 1 else 8
    return min((max(1, n // step) | 1) * step, high)


def draw(rng):
    op = rng.choice(["rec", "rec", "rec_step", "rec_grad", "rec_grad", "q8", "q8", "q8"])
    c = {"op": op, "type": rng.choice(["bf16", "f16", "bf16", "f16", "f32"])}
    if op == "q8":
        c["in"] = _channels(rng, 256, 8192)
        c["out"] = _channels(rng, 256, 16384)
        c["pair"] = rng.random() < 0.3
        most = (1 << 38) // (c["in"] * c["out"] * (2 if c["pair"] else 1))
        c["rows"] = _spread(rng, 1, min(most, 4096)) if rng.random() < 0.6 else rng.choice([1, 1, 2, 5, 8, 16, 33, 64])
        return c
    c["channels"] = _channels(rng, 240, 4096)
    if op == "rec_step":
        c["seqs"] = _spread(rng, 1, 512)
        return c
    c["seqs"] = _spread(rng, 1, 32)
    most = (1 << (27 if op == "rec" else 26)) // c["channels"]
    most = min(65536, most // (2 if c["type"] == "f32" else 1))
    c["packed"] = rng.random() < 0.6
    tokens = _spread(rng, max(64, c["seqs"]), most)
    c["tokens"] = tokens if c["packed"] else max(1, tokens // c["seqs"]) * c["seqs"]
    return c


def _lengths(case, seed):
    """Lengths of the sequences, from the seed: ragged where they are packed, an empty one and a single token among them."""
    n, total = case["seqs"], case["tokens"]
    if not case["packed"]:
        return [total // n] * n
    g = torch.Generator().manual_seed(seed)
    share = torch.rand(n, generator=g, dtype=torch.float64) + 0.05
    if n > 3:
        share[1] = 0.0
        share[2] = 0.0
    lengths = (share / share.sum() * total).floor().long()
    if n > 3:
        lengths[2] = 1
    lengths[0] += total - int(lengths.sum())
    return lengths.tolist()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = _TYPES[case["type"]]

    def normal(*shape, scale=1.0, dtype=dtype):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def uniform(low, high, *shape):
        return torch.rand(*shape, generator=g, device="cuda") * (high - low) + low

    s = {"case": case}
    if case["op"] == "q8":
        rows, k, n = case["rows"], case["in"], case["out"]
        # a few channels of the tokens stand out, as they do in such blocks
        size = torch.where(uniform(0, 1, k) < 0.01, 6.0, 1.0)
        s["x"] = (torch.randn(rows, k, generator=g, device="cuda") * size).to(dtype)
        for i in range(2 if case["pair"] else 1):
            codes = torch.randn(n, k, generator=g, device="cuda").mul_(31.0).round_().clamp_(-127, 127).to(torch.int8)
            scales = uniform(0.5, 1.5, n) / (31.0 * math.sqrt(k))
            s[f"codes{i}"], s[f"scales{i}"], s[f"bias{i}"] = codes, scales, uniform(-0.1, 0.1, n)
            if own:
                import conv2d_bias_activation_amd as c2d

                s[f"weights{i}"] = c2d.q8_pack(codes, scales)
        return s
    d, seqs = case["channels"], case["seqs"]
    if case["op"] == "rec_step":
        lead = (seqs,)
    else:
        lengths = _lengths(case, seed)
        s["max_len"], s["tokens"] = max(lengths), sum(lengths)
        s["offsets"] = torch.tensor([0] + lengths).cumsum(0).to("cuda", torch.int32)
        lead = (case["tokens"],) if case["packed"] else (seqs, case["tokens"] // seqs)
    pool = seqs if seqs == 1 else seqs + 3
    s["slots"] = torch.randperm(pool, generator=g, device="cuda")[:seqs].to(torch.int32)
    whole = normal(*lead, 3 * d)
    s["x"], s["forget"], s["gate"] = whole[..., :d], whole[..., d : 2 * d], whole[..., 2 * d :]
    s["forget_bias"] = uniform(0.0, 6.0, d)  # memories of two to some four hundred tokens
    s["state"] = normal(pool, d, scale=0.5, dtype=torch.float32)
    if case["op"] == "rec_grad":
        s["grad"] = normal(*lead, d)
        s["grad_state"] = normal(pool, d, dtype=torch.float32)
    return s


def work(case):
    e = 4 if case["type"] == "f32" else 2
    if case["op"] == "q8":
        rows, k, n, w = case["rows"], case["in"], case["out"], 2 if case["pair"] else 1
        return {"bytes": w * (n * k + 8 * n + rows * n * e) + rows * k * e, "flops": 2 * w * rows * n * k}
    d, seqs = case["channels"], case["seqs"]
    tokens = case.get("tokens", seqs)
    if case["op"] == "rec_grad":
        return {"bytes": 7 * tokens * d * e + 12 * seqs * d + 8 * d, "flops": 36 * tokens * d}
    return {"bytes": 4 * tokens * d * e + 8 * seqs * d + 4 * d, "flops": 16 * tokens * d}


def _gates(z):
    """The forget gate and what it leaves, each to full precision."""
    return 1 / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z))


def _forward(s):
    """Gates, states after each token and states before it, of all sequences as one line of tokens."""
    d = s["x"].shape[-1]
    offsets, slots = s["offsets"].long(), s["slots"].long()
    keep, take = _gates(s["forget"].reshape(-1, d).float() + s["forget_bias"])
    x = s["x"].reshape(-1, d).float()
    filled = offsets[1:] > offsets[:-1]
    starts, ends = offsets[:-1][filled], offsets[1:][filled] - 1
    start = s["state"][slots[filled]]
    h, decay = take * x, keep.clone()
    h[starts] += decay[starts] * start
    decay[starts] = 0.0
    reach = 1
    while reach < s["max_len"]:  # each token takes in what stands `reach` before it
        h[reach:] += decay[reach:] * h[:-reach]
        decay[reach:] = decay[reach:] * decay[:-reach]
        reach *= 2
    before = torch.cat([h[:1], h[:-1]])
    before[starts] = start
    return x, keep, take, h, before, starts, ends, slots[filled]


def _plain_rec(s):
    d = s["x"].shape[-1]
    _, _, _, h, _, _, ends, slots = _forward(s)
    gate = s["gate"].reshape(-1, d).float()
    y = h * (gate / (1 + torch.exp(-gate)))
    s["state"][slots] = h[ends]
    return [y.to(s["x"].dtype).reshape(s["x"].shape), s["state"]]


def _plain_step(s):
    slots = s["slots"].long()
    keep, take = _gates(s["forget"].float() + s["forget_bias"])
    h = keep * s["state"][slots] + take * s["x"].float()
    gate = s["gate"].float()
    s["state"][slots] = h
    return [(h * (gate / (1 + torch.exp(-gate)))).to(s["x"].dtype), s["state"]]


def _plain_grad(s):
    d, dtype, shape = s["x"].shape[-1], s["x"].dtype, s["x"].shape
    x, keep, take, h, before, starts, ends, slots = _forward(s)
    gate, grad = s["gate"].reshape(-1, d).float(), s["grad"].reshape(-1, d).float()
    on, off = _gates(gate)
    back = grad * gate * on
    back[ends] += s["grad_state"][slots]
    decay = torch.cat([keep[1:], keep[:1]])
    decay[ends] = 0.0
    reach = 1
    while reach < s["max_len"]:
        back[:-reach] += decay[:-reach] * back[reach:]
        decay[:-reach] = decay[:-reach] * decay[reach:]
        reach *= 2
    g_forget = back * (before - x) * (keep * take)
    g_gate = grad * h * (on * (1 + gate * off))
    s["grad_state"][slots] = keep[starts] * back[starts]
    return [*(t.to(dtype).reshape(shape) for t in (back * take, g_forget, g_gate)),
            g_forget.sum(0, dtype=torch.float64).float(), s["grad_state"]]


def _plain_q8(s):
    x = s["x"].float()
    amax = x.abs().amax(1, keepdim=True)
    scale = torch.clamp((amax.double() / torch.full_like(amax, 127.0).double()).float(), min=2.0 ** -126)
    codes = torch.round(x.double() / scale.double()).float()  # in 64 bits: exact next to the border of two codes
    out = []
    for i in range(2 if s["case"]["pair"] else 1):
        v = codes @ s[f"codes{i}"].float().t() * scale * s[f"scales{i}"] + s[f"bias{i}"]
        out.append(v.to(s["x"].dtype))
    return out


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"rec": _plain_rec, "rec_step": _plain_step, "rec_grad": _plain_grad, "q8": _plain_q8}[op](s)
    import conv2d_bias_activation_amd as c2d

    if op == "q8":
        if not s["case"]["pair"]:
            return [c2d.matmul_q8(s["x"], s["weights0"], s["bias0"])]
        rows = c2d.quantize_rows(s["x"])
        return [c2d.matmul_q8(rows, s["weights0"], s["bias0"]), c2d.matmul_q8(rows, s["weights1"], s["bias1"])]
    gates = {"gate": s["gate"], "forget_bias": s["forget_bias"], "slots": s["slots"]}
    if op == "rec_step":
        return [c2d.gated_recurrence_step(s["x"], s["forget"], state=s["state"], **gates), s["state"]]
    if s["case"]["packed"]:
        gates.update(seq_offsets=s["offsets"], longest=s["max_len"])
    if op == "rec":
        return [c2d.gated_recurrence(s["x"], s["forget"], state=s["state"], **gates), s["state"]]
    return [*c2d.gated_recurrence_backward(s["grad"], s["x"], s["forget"], state=s["state"], grad_state=s["grad_state"], **gates),
            s["grad_state"]]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "q8":
        x = s["x"].double()
        scale = (x.abs().amax(1) / torch.full((len(x),), 127.0, dtype=torch.float64, device="cuda")).float()
        scale = scale.clamp(min=2.0 ** -126).double()
        codes = torch.round(x / scale[:, None])
        out = []
        for i in range(2 if case["pair"] else 1):
            y = torch.zeros(len(x), case["out"], dtype=torch.float64, device="cuda")
            for first in range(0, case["in"], 1024):
                w = s[f"codes{i}"][:, first : first + 1024].double()
                y += torch.mm(codes[:, first : first + 1024].contiguous(), w.t().contiguous())
            out.append(y * scale[:, None] * s[f"scales{i}"].double() + s[f"bias{i}"].double())
        return out
    d, seqs = case["channels"], case["seqs"]
    step = case["op"] == "rec_step"
    offsets = list(range(seqs + 1)) if step else s["offsets"].tolist()
    length = [offsets[i + 1] - offsets[i] for i in range(seqs)]
    order = sorted(range(seqs), key=lambda i: -length[i])  # the sequences that last longest first
    first = torch.tensor([offsets[i] for i in order], device="cuda")
    last = torch.tensor([offsets[i + 1] - 1 for i in order], device="cuda")
    slots = s["slots"].long()[torch.tensor(order, device="cuda")]
    live = [sum(1 for m in length if m > t) for t in range(max(length))]
    x, gate = s["x"].double().reshape(-1, d), s["gate"].double().reshape(-1, d)
    f = torch.sigmoid(s["forget"].double().reshape(-1, d) + s["forget_bias"].double())
    state = s["state"].double()
    h = state[slots]
    after, before = torch.zeros_like(x), torch.zeros_like(x)
    for t, n in enumerate(live):  # token by token, all sequences that still have one
        at = first[:n] + t
        before[at] = h[:n]
        h[:n] = f[at] * h[:n] + (1 - f[at]) * x[at]
        after[at] = h[:n]
    if case["op"] != "rec_grad":
        state[slots] = h
        return [(after * gate * torch.sigmoid(gate)).reshape(s["x"].shape), state]
    grad = s["grad"].double().reshape(-1, d)
    carry = s["grad_state"].double()
    c = carry[slots]
    out = grad * gate * torch.sigmoid(gate)
    for t in range(len(live)):  # from each sequence's last token to its first
        n = live[t]
        at = last[:n] - t
        out[at] += c[:n]
        c[:n] = f[at] * out[at]
    carry[slots] = c
    on = torch.sigmoid(gate)
    g_forget = out * (before - x) * f * (1 - f)
    g_gate = grad * after * (on + gate * on * (1 - on))
    return [*((out * (1 - f)).reshape(s["x"].shape), g_forget.reshape(s["x"].shape), g_gate.reshape(s["x"].shape)),
            g_forget.sum(0), carry]
