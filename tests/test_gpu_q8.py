"""Rows quantized to 8 bits and their products on the GPU: codes, scales and sums exactly, outputs against 64 bits."""
import pytest
import torch

import sequence_reference as ref

pytestmark = pytest.mark.gpu

c2d = pytest.importorskip("conv2d_bias_activation_amd")
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def quantized(x):
    """Codes and scales by the definition; the 64-bit quotient of two 32-bit numbers is on the right side of every
    border between codes, from which it differs by 2^-34 of itself or not at all."""
    xd = x.double()
    finite = torch.isfinite(xd).all(1)
    s = (xd.abs().amax(1) / 127).float().clamp(min=2.0 ** -126)
    codes = torch.round(xd / s.double()[:, None]).nan_to_num(0)
    codes[~finite] = 0
    s[~finite] = float("nan")
    return codes.to(torch.int8), s


def product(codes, scales, wcodes, wscales, dtype, bias=None, alpha=None, residual=None, act="none", before=False):
    v = (codes.double() @ wcodes.double().t()) * scales.double()[:, None] * wscales.double()
    err = 3 * ref.U32 * v.abs()  # the sum to 32 bits and two products
    if bias is not None:
        v = v + bias.double()
        err = err + ref.U32 * v.abs()
    r = 0 if residual is None else residual.double()
    if before:
        v = v + r
        err = err + ref.U32 * v.abs()
    err = err * 1.001  # products of the bounds above
    y, err = ref.activate(v, err, act, alpha)
    if not before:
        y = y + r
        err = err + ref.U32 * y.abs()
    return y, ref.stored(y, err, dtype)


def _normal(seed, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def _on(t):
    return None if t is None else t.to(DEV)


def _weights(seed, n, k):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(-128, 128, (n, k), generator=g, dtype=torch.int8)
    return codes, (torch.rand(n, generator=g) + 0.5) / (74 * k ** 0.5)


def _wide(t, extra, shift):
    wide = torch.full((t.shape[0], t.shape[1] + extra + shift), float("nan"), dtype=t.dtype, device=DEV)
    view = wide[:, shift:shift + t.shape[1]]
    view.copy_(t)
    return view


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,k,extra,shift", [(1, 1, 0, 0), (3, 15, 0, 0), (16, 64, 0, 0), (17, 65, 7, 1), (5, 1000, 0, 3),
                                                (33, 2049, 1, 0), (2, 4096, 0, 0), (9, 8200, 8, 8), (2, 20011, 0, 0),
                                                (1, 131071, 0, 0)])
def test_rows(kind, rows, k, extra, shift):
    x = _normal(rows + k, rows, k, dtype=TYPES[kind])
    x[-1] *= 1e-3
    codes, scales = quantized(x)
    got_codes, got_scales = c2d.q8_unpack(c2d.quantize_rows(_wide(x, extra, shift)))
    assert torch.equal(got_scales.cpu(), scales)
    assert torch.equal(got_codes.cpu(), codes)


@pytest.mark.parametrize("kind", list(TYPES))
def test_codes_at_the_borders(kind):
    """Values on, just below and just above every border between two codes, for scales of many mantissas."""
    dtype = TYPES[kind]
    amax = (torch.rand(64, generator=torch.Generator().manual_seed(1)) * 200 + 1).to(dtype).float()
    amax[:3] = torch.tensor([127.0, 254.0, 63.5])
    s = (amax.double() / 127).float()
    border = (torch.arange(-127, 127) + 0.5).double() * s.double()[:, None]
    near = border.to(dtype)
    bits = near.view(torch.int32 if kind == "f32" else torch.int16)
    x = torch.cat([near, (bits + 1).view(dtype), (bits - 1).view(dtype), amax.to(dtype)[:, None]], 1)
    x = torch.minimum(x.float().abs(), amax[:, None]).to(dtype) * torch.sign(x)
    codes, scales = quantized(x)
    got_codes, got_scales = c2d.q8_unpack(c2d.quantize_rows(_on(x)))
    assert torch.equal(got_scales.cpu(), scales)
    assert torch.equal(got_codes.cpu(), codes)


def test_rows_at_the_ends_of_their_type():
    x = _normal(4, 12, 100)
    x[0] = 0
    x[1] = 3e-45
    x[2] *= 1e-40
    x[3, 5] = torch.finfo(torch.float32).max
    x[4, 5] = float("inf")
    x[5, 7] = float("-inf")
    x[6, 99] = float("nan")
    x[7] = -0.0
    x[8] = 2.0 ** -126
    x[9] *= 1e38
    x[10] = torch.finfo(torch.float32).max
    codes, scales = quantized(x)
    got_codes, got_scales = c2d.q8_unpack(c2d.quantize_rows(_on(x)))
    assert torch.equal(got_scales.cpu().nan_to_num(-1), scales.nan_to_num(-1))
    assert torch.equal(got_codes.cpu(), codes)
    wcodes, wscales = _weights(2, 40, 100)
    y = c2d.matmul_q8(_on(x), c2d.q8_pack(_on(wcodes), _on(wscales))).cpu()
    bad = torch.isnan(scales)  # rows 4 to 6, and 9, whose largest values are past the type
    assert bad[4:7].all() and torch.isnan(y[bad]).all()
    rest = [i for i in (0, 1, 2, 3, 7, 8, 9, 11) if not bad[i]]
    want, bound = product(codes[rest], scales[rest], wcodes, wscales, torch.float32)
    ref.close(y[rest], want, bound, "product of extreme rows")


def test_pack_and_unpack():
    for rows, k in [(1, 1), (16, 64), (17, 65), (100, 1000), (33, 4010)]:
        codes, scales = _weights(rows, rows, k)
        q = c2d.q8_pack(_on(codes), _on(scales))
        got = c2d.q8_unpack(q)
        assert torch.equal(got[0].cpu(), codes) and torch.equal(got[1].cpu(), scales)


PRODUCTS = [  # type, rows, inputs, outputs, what else
    ("bf16", 1, 1, 1, {}),
    ("f32", 1, 64, 16, {}),
    ("bf16", 1, 2048, 4096, {"bias": True}),
    ("f16", 5, 100, 33, {"bias": True, "residual": True}),
    ("bf16", 2, 8192, 1000, {"act": "silu", "bias": True}),
    ("f16", 16, 4010, 515, {"act": "relu"}),
    ("f32", 17, 129, 47, {"act": "prelu", "bias": True}),
    ("bf16", 37, 1000, 1003, {"residual": True, "before": True, "act": "relu"}),
    ("f16", 64, 320, 272, {"wide": 8}),
    ("bf16", 65, 320, 272, {"wide": 3, "shift": 1, "residual": True}),
    ("f32", 100, 777, 301, {"bias": True}),
    ("bf16", 200, 64, 4096, {}),
    ("f16", 333, 2048, 1031, {"bias": True, "act": "silu"}),
    ("bf16", 512, 4096, 512, {"bias": True, "residual": True, "act": "silu"}),
    ("bf16", 1025, 500, 700, {"bias": True, "residual": True, "act": "prelu"}),
    ("f16", 1300, 192, 1290, {}),
    ("f32", 1111, 333, 513, {"bias": True, "residual": True, "before": True, "act": "prelu", "wide": 1}),
    ("bf16", 2048, 128, 2048, {"wide": 8, "shift": 8, "residual": True}),
    ("bf16", 3001, 66, 30, {}),
    ("bf16", 3, 131071, 20, {}),
    ("f32", 90, 131071, 70, {}),
    ("f16", 1030, 20000, 260, {}),
    ("f32", 4, 8192, 100, {"bias": True, "residual": True, "act": "prelu"}),
    ("bf16", 3, 4010, 16400, {"wide": 1, "shift": 1}),
    ("f16", 1, 8191, 16391, {"residual": True, "before": True}),
    ("bf16", 4, 8193, 40, {}),
    ("f16", 2, 17, 5, {"act": "silu"}),
    # every size of tile, with rows, inputs and outputs that end inside one
    ("bf16", 333, 1000, 4090, {"bias": True, "residual": True}),
    ("f32", 340, 65, 4096, {}),
    ("f32", 4090, 70, 2039, {"act": "silu", "bias": True}),
    ("f16", 4090, 129, 2040, {"wide": 8, "bias": True}),
    ("bf16", 2040, 130, 8190, {"residual": True, "act": "relu"}),
    ("f32", 2047, 64, 8191, {"bias": True, "residual": True, "before": True, "act": "prelu"}),
]


@pytest.mark.parametrize("i", range(len(PRODUCTS)))
def test_product(i):
    kind, rows, k, n, more = PRODUCTS[i]
    dtype = TYPES[kind]
    x = _normal(i, rows, k, dtype=dtype)
    wcodes, wscales = _weights(i, n, k)
    kw = {"bias": _normal(i + 1, n, scale=0.1) if more.get("bias") else None,
          "alpha": torch.rand(n, generator=torch.Generator().manual_seed(i)) if more.get("act") == "prelu" else None,
          "residual": _normal(i + 2, rows, n, dtype=dtype) if more.get("residual") else None}
    act, before = more.get("act", "none"), more.get("before", False)
    codes, scales = quantized(x)
    want, bound = product(codes, scales, wcodes, wscales, dtype, act=act, before=before, **kw)
    extra, shift = more.get("wide", 0), more.get("shift", 0)
    weights = c2d.q8_pack(_on(wcodes), _on(wscales))
    dev = {**{name: _on(t) for name, t in kw.items()}, "act": act, "res_before_act": before}
    if kw["residual"] is not None:
        dev["residual"] = _wide(kw["residual"], extra, shift)
    y = torch.full((rows + 1, n + extra + shift), 7.0, dtype=dtype, device=DEV)
    out = y[:rows, shift:shift + n]
    xd = _wide(x, extra, shift)
    assert c2d.matmul_q8(xd, weights, out=out, **dev) is out
    ref.close(out, want, bound, f"{PRODUCTS[i]}")
    assert (y[rows] == 7).all() and (y[:, :shift] == 7).all() and (y[:, shift + n:] == 7).all()
    q = c2d.quantize_rows(xd)
    assert torch.equal(c2d.matmul_q8(q, weights, **dev), out)


def test_sums_at_their_ends():
    """The largest sums of the longest rows stay in range."""
    k = 131071
    for a, b in ((-128, -128), (-128, 127), (127, 127)):
        x = torch.full((2, k), a, dtype=torch.int8)
        w = torch.full((3, k), b, dtype=torch.int8)
        one = lambda n: torch.ones(n, device=DEV)
        y = c2d.matmul_q8(c2d.q8_pack(_on(x), one(2)), c2d.q8_pack(_on(w), one(3)))
        assert (y.cpu().double() - a * b * k).abs().max() <= ref.U32 * abs(a * b * k)


def test_scales_far_apart():
    """A product in range comes out whatever the scales' own sizes, of either side, either sign or zero."""
    codes, _ = _weights(1, 8, 200)
    wcodes, _ = _weights(2, 24, 200)
    scales = torch.tensor([1e-37, 1e36, 1.0, -2.0, 0.0, 1e-30, 3e30, float("nan")])
    wscales = torch.tensor([1e35, 1e-37, 1.0, -3.0] * 6)
    y = c2d.matmul_q8(c2d.q8_pack(_on(codes), _on(scales)), c2d.q8_pack(_on(wcodes), _on(wscales))).cpu()
    v = (codes.double() @ wcodes.double().t()) * scales.double()[:, None] * wscales.double()
    fits = v.abs() < 3e38
    normal = fits & ((v.abs() >= 2.0 ** -126) | (v == 0))
    assert torch.isnan(y[7]).all()
    off = (y.double() - v).abs()
    assert (off[normal] <= 3.003 * ref.U32 * v.abs()[normal]).all()
    assert torch.isinf(y[:7][(~fits)[:7]]).all()


def test_rows_behind_each_other_share_a_packing():
    """Products of the same rows with two weights, on two streams, from one quantization."""
    x = _normal(3, 70, 900, dtype=torch.bfloat16)
    q = c2d.quantize_rows(_on(x))
    ws = [c2d.q8_pack(*map(_on, _weights(i, 200 + i, 900))) for i in range(2)]
    want = [c2d.matmul_q8(_on(x), w) for w in ws]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ws]
    got = [c2d.matmul_q8(q, w, stream=s) for w, s in zip(ws, streams)]
    own = [c2d.matmul_q8(_on(x), w, stream=s) for w, s in zip(ws, streams)]
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, own):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("rows", [1, 40, 300, 1500])
def test_captured_product_replays(rows):
    x, x2 = _on(_normal(5, rows, 700, dtype=torch.bfloat16)), _on(_normal(6, rows, 700, dtype=torch.bfloat16))
    w = c2d.q8_pack(*map(_on, _weights(7, 900, 700)))
    want = [c2d.matmul_q8(t, w) for t in (x, x2)]
    held, y = x.clone(), torch.empty(rows, 900, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(4 << 20, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c2d.matmul_q8(held, w, out=y, workspace=ws)
    for i in (0, 1, 0, 1):
        held.copy_((x, x2)[i])
        y.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])


def test_offsets_past_32_bits():
    """Rows so far apart that an element's index passes 2^31."""
    rows, k, n, pitch = 300, 64, 32, 1 << 23
    whole = torch.empty(rows * pitch + 256, dtype=torch.bfloat16, device=DEV)
    view = lambda first, d: whole[first:first + rows * pitch].view(rows, pitch)[:, :d]
    x, r = _on(_normal(1, rows, k, dtype=torch.bfloat16)), _on(_normal(2, rows, n, dtype=torch.bfloat16))
    view(0, k).copy_(x)
    view(128, n).copy_(r)
    w = c2d.q8_pack(*map(_on, _weights(3, n, k)))
    want = c2d.matmul_q8(x, w, residual=r)
    assert torch.equal(c2d.matmul_q8(view(0, k), w, residual=view(128, n)), want)
    out = torch.empty(rows * pitch, dtype=torch.bfloat16, device=DEV).view(rows, pitch)[:, :n]
    c2d.matmul_q8(x, w, residual=r, out=out)
    assert torch.equal(out, want)


def test_packed_rows_past_2_gib():
    """Weights whose packed bytes pass 2^31: their last rows, and the outputs that read them."""
    n, k, tail = 140001, 16384, 40
    g = torch.Generator(device=DEV).manual_seed(11)
    w = torch.randn(n, k, generator=g, device=DEV, dtype=torch.bfloat16)
    weights = c2d.quantize_rows(w)
    assert weights.data.numel() > 1 << 31
    wcodes, wscales = quantized(w[-tail:].cpu())
    codes, scales = c2d.q8_unpack(weights)
    assert torch.equal(codes[-tail:].cpu(), wcodes) and torch.equal(scales[-tail:].cpu(), wscales)
    again = c2d.q8_pack(codes, scales)
    assert torch.equal(again.data, weights.data)
    del again, codes, w
    for rows in (1, 30, 600):
        x = _normal(rows, rows, k, dtype=torch.bfloat16)
        want, bound = product(*quantized(x), wcodes, wscales, torch.bfloat16)
        y = c2d.matmul_q8(_on(x), weights)
        ref.close(y[:, -tail:], want, bound, f"{rows} rows")


def test_product_needs_a_workspace_or_packed_rows():
    x = _on(_normal(1, 20, 64))
    w = c2d.q8_pack(*map(_on, _weights(1, 8, 64)))
    with pytest.raises(c2d.Conv2dError, match="needs a workspace"):
        c2d.matmul_q8(x, w, workspace=False)
    assert torch.equal(c2d.matmul_q8(x[:4], w, workspace=False), c2d.matmul_q8(x, w)[:4])  # a few rows need none
    with pytest.raises(ValueError, match="inputs"):
        c2d.matmul_q8(c2d.quantize_rows(x[:, :32]), w)
    assert c2d.matmul_q8(x[:0], w).shape == (0, 8)
    assert c2d.matmul_q8(c2d.quantize_rows(x[:0]), w).shape == (0, 8)
