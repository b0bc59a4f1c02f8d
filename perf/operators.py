"""Cases of the sequence operators: short causal convolution and selective state space scan, for prompts and for
single tokens, and products of a few token rows with 4-bit weights.

``run`` computes a case with the library's operators where ``own`` is true, and otherwise in plain 32-bit torch
operations. ``exact`` computes the definition in 64 bits, one token at a time.

The sizes are those of a served state-space block of 240 to 8192 channels: projections make the 2*D columns "x | gate"
and the columns "B | C" that the operators read as slices, sequences of a batch have different lengths (empty ones
and single tokens among them), and states live in a pool whose rows the sequences name.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # a short prompt of one user, on the narrow block: latency
        {"name": "conv prompt short", "op": "conv", "type": "f16", "seqs": 1, "tokens": 77, "channels": 512, "width": 4, "packed": False},
        # a prefill batch of ragged prompts, packed, on a wide block
        {"name": "conv prompt batch", "op": "conv", "type": "bf16", "seqs": 16, "tokens": 32768, "channels": 4096, "width": 4, "packed": True},
        # one user's next token
        {"name": "conv token one", "op": "conv_step", "type": "bf16", "seqs": 1, "channels": 2048, "width": 4},
        # a full decode batch
        {"name": "conv token batch", "op": "conv_step", "type": "f16", "seqs": 384, "channels": 4096, "width": 3},
        # a small block in 32 bits with many states and odd lengths
        {"name": "scan prompt f32", "op": "scan", "type": "f32", "seqs": 3, "tokens": 999, "channels": 240, "states": 64, "groups": 2, "packed": True},
        # one long document: few channels' worth of work, many tokens
        {"name": "scan prompt long", "op": "scan", "type": "bf16", "seqs": 1, "tokens": 32768, "channels": 1024, "states": 16, "groups": 1, "packed": False},
        # a prefill batch of ragged prompts, packed, on a wide block
        {"name": "scan prompt batch", "op": "scan", "type": "bf16", "seqs": 24, "tokens": 16384, "channels": 4096, "states": 16, "groups": 1, "packed": True},
        # one user's next token
        {"name": "scan token one", "op": "scan_step", "type": "bf16", "seqs": 1, "channels": 2048, "states": 16, "groups": 1},
        # a full decode batch
        {"name": "scan token batch", "op": "scan_step", "type": "f16", "seqs": 512, "channels": 4096, "states": 16, "groups": 1},
        # a projection of one user's token
        {"name": "w4 one row", "op": "w4", "type": "bf16", "rows": 1, "in": 2048, "out": 4096, "group": 128, "zeros": False},
        # the same for a few users, odd sizes: the last group and the last tile are partial
        {"name": "w4 odd", "op": "w4", "type": "f16", "rows": 5, "in": 4010, "out": 10007, "group": 32, "zeros": True},
        # a wide output projection for a decode batch
        {"name": "w4 wide", "op": "w4", "type": "bf16", "rows": 16, "in": 8192, "out": 32768, "group": 64, "zeros": True},
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
    odd = max(1, n // step) | 1
    return min(odd * step, high)


def draw(rng):
    op = rng.choice(["conv", "conv_step", "scan", "scan_step", "w4"])
    c = {"op": op, "type": rng.choice(["bf16", "f16", "bf16", "f16", "f32"])}
    if op == "w4":
        c["type"] = rng.choice(["bf16", "f16"])
        c["rows"] = rng.choice([1, 1, 2, 3, 4, 7, 8, 13, 16])
        c["in"] = _channels(rng, 256, 8192)
        c["out"] = _channels(rng, 256, 32768)
        c["group"] = rng.choice([32, 64, 128])
        c["zeros"] = rng.random() < 0.5
        return c
    c["channels"] = _channels(rng, 240, 4096)
    if op in ("conv", "conv_step"):
        c["width"] = rng.choice([2, 3, 4, 4])
    else:
        c["states"] = rng.choice([8, 16, 16, 16, 24, 64])
        c["groups"] = rng.choice([g for g in (1, 1, 2, 4, 8) if c["channels"] % g == 0])
    if op in ("conv_step", "scan_step"):
        most = 512 if op == "conv_step" else max(1, 512 * 4096 * 16 // (c["channels"] * c["states"]))
        c["seqs"] = _spread(rng, 1, min(512, most))
        return c
    c["seqs"] = _spread(rng, 1, 32)
    most = (32768 * 4096 if op == "conv" else 16384 * 4096 * 16 // c["states"]) // c["channels"]
    most = min(32768, most // (2 if c["type"] == "f32" else 1))
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
    if case["op"] == "w4":
        rows, k, n, group = case["rows"], case["in"], case["out"], case["group"]
        groups = -(-k // group)
        s["x"] = normal(rows, k)
        s["codes"] = torch.randint(0, 256, (n, (k + 1) // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["scales"] = (uniform(0.5, 1.5, n, groups) / (4.6 * math.sqrt(k))).to(dtype)
        s["zeros"] = torch.randint(6, 11, (n, groups), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
        s["bias"] = uniform(-0.1, 0.1, n)
        s["residual"] = normal(rows, n)
        if own:
            import conv2d_bias_activation_amd as c2d

            s["weights"] = c2d.w4_pack(s["codes"], s["scales"], s["zeros"], in_features=k, group=group)
        return s
    d = case["channels"]
    seqs = case["seqs"]
    step = case["op"].endswith("_step")
    if step:
        lead = (seqs,)
    else:
        lengths = _lengths(case, seed)
        s["max_len"] = max(lengths)
        s["tokens"] = sum(lengths)
        starts = torch.tensor([0] + lengths).cumsum(0)
        s["offsets"] = starts.to("cuda", torch.int32)
        lead = (case["tokens"],) if case["packed"] else (seqs, case["tokens"] // seqs)
    pool = seqs if seqs == 1 else seqs + 3
    s["slots"] = torch.randperm(pool, generator=g, device="cuda")[:seqs].to(torch.int32)
    both = normal(*lead, 2 * d)
    s["x"], s["gate"] = both[..., :d], both[..., d:]
    if case["op"].startswith("conv"):
        width = case["width"]
        s["w"] = normal(d, width, scale=1 / math.sqrt(width))
        s["bias"] = uniform(-0.1, 0.1, d)
        s["state"] = normal(pool, width - 1, d)
        return s
    n, groups = case["states"], case["groups"]
    bc = normal(*lead, 2 * groups * n)
    s["B"] = bc[..., : groups * n].unflatten(-1, (groups, n))
    s["C"] = bc[..., groups * n :].unflatten(-1, (groups, n))
    s["dt"] = normal(*lead, d, scale=0.5)
    first = torch.exp(uniform(math.log(0.001), math.log(0.1), d))  # step sizes at rest, as such blocks are initialised
    s["dt_bias"] = first + torch.log(-torch.expm1(-first))
    s["A"] = -torch.arange(1, n + 1, device="cuda", dtype=torch.float32).expand(d, n) * uniform(0.8, 1.25, d, n)
    s["skip"] = uniform(0.5, 1.5, d)
    s["state"] = normal(pool, d, n, scale=0.5, dtype=torch.float32)
    return s


def work(case):
    e = 4 if case["type"] == "f32" else 2
    if case["op"] == "w4":
        rows, k, n = case["rows"], case["in"], case["out"]
        groups = -(-k // case["group"])
        return {"bytes": n * k / 2 + n * groups * (e + (1 if case["zeros"] else 0)) + rows * (k + 2 * n) * e + 4 * n,
                "flops": 2 * rows * n * k}
    d, seqs = case["channels"], case["seqs"]
    tokens = case.get("tokens", seqs)
    if case["op"].startswith("conv"):
        w = case["width"]
        return {"bytes": 2 * tokens * d * e + 2 * seqs * (w - 1) * d * e + d * (w * e + 4), "flops": 2 * tokens * d * w}
    n = case["states"]
    return {"bytes": 4 * tokens * d * e + 2 * tokens * case["groups"] * n * e + 8 * seqs * d * n + d * (4 * n + 8),
            "flops": 7 * tokens * d * n}


def _places(s):
    """For each token its sequence and its place in it, and the sequences' lengths."""
    offsets = s["offsets"].long()
    at = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(offsets, at, right=True) - 1
    return seq, at - offsets[seq], offsets[1:] - offsets[:-1], offsets


def _plain_conv(s):
    x, w, state = s["x"], s["w"].float(), s["state"]
    d, width = w.shape
    seq, place, length, offsets = _places(s)
    slots = s["slots"].long()
    tokens = x.reshape(-1, d).float()
    old = state[slots].float()  # [seqs, width - 1, d]
    rows = torch.cat([tokens, old.reshape(-1, d)])
    back = torch.arange(width - 1, -1, -1, device="cuda")  # how far back each tap lies
    at = torch.arange(s["tokens"], device="cuda")
    before = s["tokens"] + seq[:, None] * (width - 1) + width - 1 + place[:, None] - back
    source = torch.where(place[:, None] >= back, at[:, None] - back, before)
    y = s["bias"].expand(s["tokens"], d)
    for j in range(width):  # taps
        y = y + rows[source[:, j]] * w[:, j]
    y = y / (1 + torch.exp(-y))
    kept = length[:, None] - back[:-1]  # places of the last width - 1 inputs
    first = s["tokens"] + torch.arange(len(slots), device="cuda")[:, None] * (width - 1)
    source = torch.where(kept >= 0, offsets[:-1, None] + kept, first + width - 1 + kept)
    state[slots] = rows[source].to(state.dtype)
    return [y.to(x.dtype).reshape(x.shape), state]


def _plain_conv_step(s):
    x, w, state, slots = s["x"], s["w"].float(), s["state"], s["slots"].long()
    line = torch.cat([state[slots], x[:, None]], 1)
    y = (line.float() * w.t()).sum(1) + s["bias"]
    state[slots] = line[:, 1:]
    return [(y / (1 + torch.exp(-y))).to(x.dtype), state]


def _plain_scan_step(s):
    u, state, slots = s["x"], s["state"], s["slots"].long()
    d, n = s["A"].shape
    groups = s["B"].shape[-2]
    x, gate = u.float(), s["gate"].float()
    step = s["dt"].float() + s["dt_bias"]
    step = torch.clamp(step, min=0) + torch.log1p(torch.exp(-step.abs()))
    b = s["B"].float().repeat_interleave(d // groups, 1)
    c = s["C"].float().repeat_interleave(d // groups, 1)
    h = state[slots] * torch.exp(step[:, :, None] * s["A"]) + (step * x)[:, :, None] * b
    y = (h * c).sum(-1) + s["skip"] * x
    state[slots] = h
    return [(y * (gate / (1 + torch.exp(-gate)))).to(u.dtype), state]


def _plain_scan(s):
    u, state = s["x"], s["state"]
    d, n = s["A"].shape
    groups = s["B"].shape[-2]
    seq, place, length, offsets = _places(s)
    slots = s["slots"].long()
    x = u.reshape(-1, d).float()
    step = s["dt"].reshape(-1, d).float() + s["dt_bias"]
    step = torch.clamp(step, min=0) + torch.log1p(torch.exp(-step.abs()))
    per = d // groups
    b = s["B"].reshape(-1, groups, 1, n).float()
    c = s["C"].reshape(-1, groups, 1, n).float()
    decay = torch.exp(step[:, :, None] * s["A"])
    h = ((step * x).reshape(-1, groups, per, 1) * b).reshape(-1, d, n)
    filled = length > 0
    starts = offsets[:-1][filled]
    h[starts] += decay[starts] * state[slots[filled]]
    decay[starts] = 0.0
    reach = 1
    while reach < s["tokens"] and reach < s["max_len"]:  # each token takes in what stands `reach` before it
        h[reach:] += decay[reach:] * h[:-reach]
        decay[reach:] = decay[reach:] * decay[:-reach]
        reach *= 2
    y = (h.reshape(-1, groups, per, n) * c).sum(-1).reshape(-1, d) + s["skip"] * x
    gate = s["gate"].reshape(-1, d).float()
    y = y * (gate / (1 + torch.exp(-gate)))
    state[slots[filled]] = h[offsets[1:][filled] - 1]
    return [y.to(u.dtype).reshape(u.shape), state]


def _plain_w4(s):
    case, x = s["case"], s["x"]
    codes = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).flatten(1)[:, : case["in"]].float()
    zeros = 8.0 if s["zeros"] is None else s["zeros"].float().repeat_interleave(case["group"], 1)[:, : case["in"]]
    scales = s["scales"].float().repeat_interleave(case["group"], 1)[:, : case["in"]]
    y = x.float() @ ((codes - zeros) * scales).t() + s["bias"] + s["residual"].float()
    return [y.to(x.dtype)]


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"conv": _plain_conv, "conv_step": _plain_conv_step, "scan": _plain_scan, "scan_step": _plain_scan_step, "w4": _plain_w4}[op](s)
    import conv2d_bias_activation_amd as c2d

    if op == "w4":
        return [c2d.matvec_w4(s["x"], s["weights"], s["bias"], residual=s["residual"])]
    if op == "conv_step":
        return [c2d.causal_conv1d_step(s["x"], s["w"], s["bias"], state=s["state"], slots=s["slots"], act="silu"), s["state"]]
    if op == "scan_step":
        y = c2d.selective_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], state=s["state"], skip=s["skip"], gate=s["gate"],
                                    dt_bias=s["dt_bias"], softplus=True, slots=s["slots"])
        return [y, s["state"]]
    packed = {"seq_offsets": s["offsets"]} if s["case"]["packed"] else {}
    if op == "conv":
        return [c2d.causal_conv1d(s["x"], s["w"], s["bias"], state=s["state"], slots=s["slots"], act="silu", **packed), s["state"]]
    y = c2d.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], state=s["state"], skip=s["skip"], gate=s["gate"],
                           dt_bias=s["dt_bias"], softplus=True, slots=s["slots"], longest=s["max_len"], **packed)
    return [y, s["state"]]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "w4":
        k, group = case["in"], case["group"]
        y = s["bias"].double() + s["residual"].double()
        for first in range(0, k, group):  # group by group
            last = min(k, first + group)
            at = torch.arange(first, last, device="cuda")
            codes = ((s["codes"][:, at // 2].int() >> (4 * (at % 2))) & 15).double()
            zero = 8.0 if s["zeros"] is None else s["zeros"][:, first // group, None].double()
            w = (codes - zero) * s["scales"][:, first // group, None].double()
            y += torch.mm(s["x"][:, first:last].double(), w.t().contiguous())
        return [y]
    offsets = s["offsets"].tolist() if "offsets" in s else list(range(case["seqs"] + 1))
    d = case["channels"]
    tokens = s["x"].double().reshape(-1, d)
    state = s["state"].double()
    y = torch.zeros_like(tokens)
    if case["op"].startswith("conv"):
        width = case["width"]
        w, bias = s["w"].double(), s["bias"].double()
        for i, slot in enumerate(s["slots"].tolist()):  # sequence by sequence
            line = torch.cat([state[slot], tokens[offsets[i] : offsets[i + 1]]])
            if offsets[i + 1] > offsets[i]:
                v = (line.unfold(0, width, 1) * w).sum(-1) + bias
                y[offsets[i] : offsets[i + 1]] = v * torch.sigmoid(v)
            state[slot] = line[len(line) - (width - 1) :]
        return [y.reshape(s["x"].shape), state]
    n, groups = case["states"], case["groups"]
    dt = torch.logaddexp(s["dt"].double().reshape(-1, d) + s["dt_bias"].double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    gate = s["gate"].double().reshape(-1, d)
    bs, cs = (s[k].double().reshape(-1, groups, n) for k in "BC")
    a, skip = s["A"].double(), s["skip"].double()
    length = [offsets[i + 1] - offsets[i] for i in range(case["seqs"])]
    slots = s["slots"].long()
    first = torch.tensor(offsets[:-1], device="cuda")
    h = state[slots]
    for t in range(max(length)):  # token by token, all sequences that still have one
        live = [i for i, m in enumerate(length) if m > t]
        some = torch.tensor(live, device="cuda") if len(live) < len(length) else slice(None)
        at = first[some] + t
        x, step = tokens[at], dt[at]
        b = bs[at].repeat_interleave(d // groups, 1)
        c = cs[at].repeat_interleave(d // groups, 1)
        now = h[some] * torch.exp(step[:, :, None] * a) + (step * x)[:, :, None] * b
        h[some] = now
        z = gate[at]
        y[at] = ((now * c).sum(-1) + skip * x) * z * torch.sigmoid(z)
    state[slots] = h
    return [y.reshape(s["x"].shape), state]
