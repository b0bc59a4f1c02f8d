"""A served state-space block: a prompt in one pass, then tokens one at a time.

The block is x + out(scan(conv(in(x)))): a projection to "value | gate" columns, the short
causal convolution, projections to the step size and to the columns "B | C", the selective
scan with its gate, and a projection back added to x. Its projections have 4-bit weights. A
prompt's go through the library's 1x1 convolution (`conv2d_fused`, on the weights' values in
bf16, laid out once); a token's are products with the 4-bit weights themselves (`matvec_w4`),
which reads a quarter of the bytes. A token step is recorded once into a HIP graph and
replayed; the states move on in place.

    python examples/state_space_block.py [--model 1024] [--prompt 2048] [--tokens 64] [--batch 4]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import conv2d_bias_activation_amd as c2d  # noqa: E402


class Projection:
    """Random 4-bit weights [out, in], as matvec_w4 and as conv2d_fused take them."""

    def __init__(self, out_features, in_features, generator, group=32):
        dev = generator.device
        codes = torch.randint(0, 256, (out_features, (in_features + 1) // 2), generator=generator, device=dev, dtype=torch.uint8)
        groups = -(-in_features // group)
        scales = ((torch.rand(out_features, groups, generator=generator, device=dev) + 0.5) / (4.6 * in_features ** 0.5)).bfloat16()
        self.w4 = c2d.w4_pack(codes, scales, in_features=in_features, group=group)
        q = torch.stack([codes & 15, codes >> 4], -1).flatten(1)[:, :in_features].float() - 8
        w = (q * scales.float().repeat_interleave(group, 1)[:, :in_features]).bfloat16()
        self.ohwi = w.reshape(out_features, 1, 1, in_features)

    def prompt(self, x, residual=None):
        """x [tokens, in], contiguous."""
        r = None if residual is None else residual[None, None]
        return c2d.conv2d_fused(x[None, None], self.ohwi, residual=r)[0, 0]

    def token(self, x, residual=None):
        """x [rows, in], rows at any stride."""
        return c2d.matvec_w4(x, self.w4, residual=residual)


class StateSpaceBlock:
    def __init__(self, model, batch, inner=None, states=16, rank=32, width=4, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        inner = inner or 2 * model
        self.inner, self.states, self.rank = inner, states, rank
        self.into = Projection(2 * inner, model, g)
        self.steps = Projection(rank + 2 * states, inner, g)
        self.dt = Projection(inner, rank, g)
        self.out = Projection(model, inner, g)
        self.conv_w = (torch.randn(inner, width, generator=g, device=device) / width ** 0.5).bfloat16()
        self.conv_b = torch.zeros(inner, device=device)
        first = 0.001 * 100 ** torch.rand(inner, generator=g, device=device)
        self.scan = {"skip": torch.ones(inner, device=device), "dt_bias": first + torch.log(-torch.expm1(-first)),
                     "softplus": True}
        self.A = -torch.arange(1, states + 1, device=device, dtype=torch.float32).repeat(inner, 1)
        # the states of `batch` sequences
        self.conv_state = torch.zeros(batch, width - 1, inner, device=device, dtype=torch.bfloat16)
        self.scan_state = torch.zeros(batch, inner, states, device=device)

    def _split(self, steps):
        b = steps[:, self.rank:].unflatten(-1, (2, 1, self.states))
        return steps[:, :self.rank], b[:, 0], b[:, 1]

    def prompt(self, x, lengths, slots, fresh=True):
        """x [tokens, model], the sequences packed; their states end in the rows `slots`."""
        offsets = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).to(x.device)
        packed = {"seq_offsets": offsets, "slots": slots, "fresh": fresh}
        both = self.into.prompt(x)
        v = c2d.causal_conv1d(both[:, :self.inner], self.conv_w, self.conv_b, act="silu", state=self.conv_state, **packed)
        low, b, c = self._split(self.steps.prompt(v))
        y = c2d.selective_scan(v, self.dt.prompt(low.contiguous()), self.A, b, c, gate=both[:, self.inner:],
                               state=self.scan_state, longest=max(lengths), **self.scan, **packed)
        return self.out.prompt(y, residual=x)

    def token(self, x):
        """x [batch, model]: the next token of every sequence."""
        both = self.into.token(x)
        v = c2d.causal_conv1d_step(both[:, :self.inner], self.conv_w, self.conv_b, act="silu", state=self.conv_state)
        low, b, c = self._split(self.steps.token(v))
        y = c2d.selective_scan_step(v, self.dt.token(low), self.A, b, c, gate=both[:, self.inner:], state=self.scan_state,
                                    **self.scan)
        return self.out.token(y, residual=x)

    def record(self, batch, model):
        """(graph, its input, its output) of a token step. The warm-up's traces in the states are taken back."""
        x = torch.zeros(batch, model, device=self.A.device, dtype=torch.bfloat16)
        kept = self.conv_state.clone(), self.scan_state.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.token(x)
        torch.cuda.current_stream().wait_stream(side)
        self.conv_state.copy_(kept[0])
        self.scan_state.copy_(kept[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = self.token(x)
        return graph, x, y


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--model", type=int, default=1024)
    ap.add_argument("--prompt", type=int, default=2048)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--batch", type=int, default=4)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(1)
    lengths = [max(1, a.prompt - 37 * i) for i in range(a.batch)]
    after = [torch.randn(n + a.tokens, a.model, generator=g, device="cuda").bfloat16() for n in lengths]
    slots = torch.arange(a.batch, device="cuda", dtype=torch.int32)
    block = StateSpaceBlock(a.model, a.batch)

    # everything as one prompt
    whole = block.prompt(torch.cat(after), [len(x) for x in after], slots).split([len(x) for x in after])
    states = block.conv_state.clone(), block.scan_state.clone()

    # the prompt, then token by token
    prompt = torch.cat([x[:n] for x, n in zip(after, lengths)])
    block.prompt(prompt, lengths, slots)
    graph, x, y = block.record(a.batch, a.model)
    worst = 0.0
    for t in range(a.tokens):
        x.copy_(torch.stack([s[n + t] for s, n in zip(after, lengths)]))
        graph.replay()
        want = torch.stack([w[n + t] for w, n in zip(whole, lengths)]).float()
        worst = max(worst, float((y.float() - want).norm() / want.norm()))
    drift = [float((s.float() - w.float()).norm() / w.float().norm()) for s, w in
             zip((block.conv_state, block.scan_state), states)]

    def timed(call, reps):
        call()
        torch.cuda.synchronize()
        start = time.perf_counter()
        for _ in range(reps):
            call()
        torch.cuda.synchronize()
        return (time.perf_counter() - start) / reps * 1e6

    us_prompt = timed(lambda: block.prompt(prompt, lengths, slots), 10)
    us_token = timed(graph.replay, 100)
    us_eager = timed(lambda: block.token(x), 100)
    print(f"{a.batch} prompts, {len(prompt)} tokens x {a.model}: {us_prompt:.0f} us ({len(prompt) / us_prompt:.2f} tokens/us)")
    print(f"{a.batch} next tokens: {us_token:.1f} us in a graph, {us_eager:.1f} us call by call")
    print(f"tokens against one prompt: outputs {worst:.1e}, states {drift[0]:.1e} and {drift[1]:.1e} apart (relative)")
    return worst, drift


if __name__ == "__main__":
    main()
