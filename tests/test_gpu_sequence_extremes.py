"""Causal convolution, selective scan and 4-bit products with values at the ends of their types, against their
definitions in 64 bits."""
import pytest
import torch

import sequence_reference as ref
from test_gpu_sequence import DEV, _normal, _on, _reference, _rng, _scan_args, _scan_case

pytestmark = pytest.mark.gpu

c2d = pytest.importorskip("conv2d_bias_activation_amd")


# type, lengths, packed, channels, states, groups: every number of states that has a kernel of its own, ends inside a
# tile, sequences that are split and that are not
FAST = [("f32", [37], False, 64, 16, 1), ("bf16", [33, 0, 1, 2, 70, 17], True, 72, 16, 1), ("f16", [13], False, 40, 3, 1),
        ("f32", [21, 9], True, 36, 6, 2), ("f32", [29], False, 20, 32, 1), ("bf16", [19], False, 24, 50, 1),
        ("f32", [15, 3], True, 16, 100, 1), ("f32", [11], False, 8, 200, 1), ("f32", [901], False, 64, 16, 1),
        ("bf16", [1001, 5, 700], True, 40, 8, 1), ("f32", [603], False, 24, 64, 2)]


@pytest.mark.parametrize("kind,lengths,packed,d,n,groups", FAST)
@pytest.mark.parametrize("rate", [-float("inf"), -3e38])
def test_rates_without_bounds(rate, kind, lengths, packed, d, n, groups):
    """A state whose rate A is infinite, or so large that A log2(e) is, forgets at once: exp(d A) is zero for every
    step of these sequences, so the definition's values are those of A = -1e30."""
    c = _scan_case(61, kind, lengths, d, n, groups, {})
    c["A"] = c["A"].clone()
    c["A"][:, ::3] = -1e30
    want, bound, state, state_bound = _reference(c, lengths)
    c["A"][:, ::3] = rate
    _, args, kw = _scan_args(c, lengths, packed, {})
    for workspace in (None, False):
        dev_state = _on(c["state"])
        y = c2d.selective_scan(*args, **kw, state=dev_state, longest=max(lengths), workspace=workspace)
        ref.close(y.reshape(-1, d), want, bound, "y")
        ref.close(dev_state, state, state_bound, "state")


@pytest.mark.parametrize("n", [4, 5, 16, 64, 130])
def test_token_rates_without_bounds(n):
    c = _scan_case(62, "f32", [1] * 3, 48, n, 1, {})
    c["A"] = c["A"].clone()
    c["A"][:, ::2] = -1e30
    want, bound, state, state_bound = _reference(c, [1] * 3)
    for rate in (-float("inf"), -3e38):
        c["A"][:, ::2] = rate
        _, args, kw = _scan_args(c, [1] * 3, True, {})
        del kw["seq_offsets"]
        dev_state = _on(c["state"])
        ref.close(c2d.selective_scan_step(*args, **kw, state=dev_state), want, bound, "y")
        ref.close(dev_state, state, state_bound, "state")


@pytest.mark.parametrize("lengths,n", [([45], 16), ([700], 16), ([21], 5)])
def test_empty_steps_keep_the_largest_finite_rates(lengths, n):
    """exp(0 A) = 1 for any finite A: a token without a step leaves the state as it is."""
    c = _scan_case(63, "f32", lengths, 64, n, 1, {"plain": True})
    c["A"] = c["A"].clone()
    c["A"][:, ::2] = -3.4e38
    c["dt"][2:] = 0.0
    want, bound, state, state_bound = _reference(c, lengths)
    _, args, kw = _scan_args(c, lengths, False, {})
    for workspace in (None, False):
        dev_state = _on(c["state"])
        y = c2d.selective_scan(*args, **kw, state=dev_state, workspace=workspace)
        ref.close(y.reshape(-1, 64), want, bound, "y")
        ref.close(dev_state, state, state_bound, "state")
    c = _scan_case(64, "f32", [1] * 2, 64, n, 1, {"plain": True})
    c["A"] = c["A"].clone()
    c["A"][:, 1::2] = -3.4e38
    c["dt"][:] = 0.0
    want, bound, state, state_bound = _reference(c, [1] * 2)
    _, args, kw = _scan_args(c, [1] * 2, True, {})
    del kw["seq_offsets"]
    dev_state = _on(c["state"])
    ref.close(c2d.selective_scan_step(*args, **kw, state=dev_state), want, bound, "y")
    ref.close(dev_state, state, state_bound, "state")


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("size", [1e-37, 1e-30, 2e38])
@pytest.mark.parametrize("rows,k,n,group", [(1, 256, 64, 128), (5, 401, 130, 32), (17, 640, 48, 64)])
def test_products_of_the_largest_and_smallest_rows(rows, k, n, group, size, zeros):
    """bf16 reaches from 1e-38 to 3e38. Rows of values near either end give finite products and, as the scales bring
    them back to moderate numbers, the definition's."""
    g = _rng(66)
    x = (torch.rand(rows, k, generator=g) * 0.5 + 0.5) * size * torch.sign(torch.randn(rows, k, generator=g))
    if size > 1:  # sums of the products themselves stay in range: one large value for each group
        x = torch.where(torch.arange(k) % group == 3, x / 15, x * 2.0 ** -40)
    x = x.bfloat16()
    groups = -(-k // group)
    codes = torch.randint(0, 256, (n, (k + 1) // 2), generator=g, dtype=torch.uint8)
    scales = ((torch.rand(n, groups, generator=g) + 0.5) / size).bfloat16()
    z = torch.randint(0, 16, (n, groups), generator=g, dtype=torch.uint8) if zeros else None
    want, bound = ref.w4(x, codes, scales, z, group, None, None, None, "none", False)
    # a product below fp32's smallest normal number may be off by half of its smallest step, 2^-150, times the scale, or by
    # 2^12 as much where codes are taken times 2^-12
    bound = bound + k * 2.0 ** -138 * scales.double().max()
    weights = c2d.w4_pack(_on(codes), _on(scales), _on(z), in_features=k, group=group)
    ref.close(c2d.matvec_w4(_on(x), weights), want, bound, "w4")


@pytest.mark.parametrize("d", [40, 64])
def test_growth_past_a_chunk(d):
    """Steps may be negative or rates positive. A state that is zero stays so however far the decay of a whole chunk
    passes fp32's range, and one that grows and shrinks again by e^96 keeps its value."""
    tokens, n = 900, 16
    c = _scan_case(65, "f32", [tokens], d, n, 1, {"plain": True})
    c["A"] = torch.ones(d, n)
    place = torch.arange(tokens)
    c["dt"] = torch.where(place // 32 % 2 == 0, 3.0, -3.0)[:, None].repeat(1, d)  # a sum of 96 in 32 tokens
    c["dt"][896:] = 0.125
    c["u"][:896] = 0.0
    c["state"] = torch.full((1, d, n), 1e-36)
    c["state"][:, ::2] = 0.0
    want, bound, state, state_bound = _reference(c, [tokens])
    assert all(torch.isfinite(t).all() for t in (want, bound, state, state_bound))
    _, args, kw = _scan_args(c, [tokens], False, {})
    for workspace in (False, None):
        dev_state = _on(c["state"])
        y = c2d.selective_scan(*args, **kw, state=dev_state, workspace=workspace)
        ref.close(y.reshape(-1, d), want, bound, "y")
        ref.close(dev_state, state, state_bound, "state")


@pytest.mark.parametrize("count,n,groups", [(70, 4, 1), (256, 4, 1), (256, 16, 2), (130, 64, 1)])
def test_many_whole_sequences(count, n, groups):
    """Sequences taken in the order of their lengths, equal and empty ones among them, in every number that is ordered."""
    lengths = torch.randint(0, 140, (count,), generator=_rng(67)).tolist()
    lengths[3] = lengths[count - 1] = max(lengths)
    d = 32
    assert 4 * sum(lengths) >= count * count
    c = _scan_case(68, "f32", lengths, d, n, groups, {})
    c["slots"] = torch.randperm(count + 2, generator=_rng(69))[:count].to(torch.int32)
    want, bound, state, state_bound = _reference(c, lengths)
    _, args, kw = _scan_args(c, lengths, True, {})
    dev_state = _on(c["state"])
    ref.close(c2d.selective_scan(*args, **kw, state=dev_state, workspace=False), want, bound, "y")
    ref.close(dev_state, state, state_bound, "state")
