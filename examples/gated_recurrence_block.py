"""A gated-recurrence block with 8-bit weights, served, and the recurrence's gradient in a training step.

The block is x + out(recurrence(conv(into(x)), gate(x))): the token rows are quantized to 8
bits once for two projections, to the columns "value | forget" and to the gate, then come the
short causal convolution of the values, the gated linear recurrence with its gate, and a
projection back, added to x. Prompts and single tokens take the same 8-bit weights, so both
see the same codes. A token step is recorded once into a HIP graph and replayed; the states
move on in place.

`recurrence` is the same operator as a function that torch differentiates, for training.

    python examples/gated_recurrence_block.py [--model 1024] [--prompt 2048] [--tokens 64] [--batch 4]
"""
import argparse
import os
import sys
import time

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import conv2d_bias_activation_amd as c2d  # noqa: E402


class _Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, forget, gate, forget_bias):
        ctx.save_for_backward(x, forget, gate, forget_bias)
        return c2d.gated_recurrence(x, forget, gate=gate, forget_bias=forget_bias)

    @staticmethod
    @once_differentiable  # the library has no gradient of the gradient
    def backward(ctx, grad):
        x, forget, gate, forget_bias = ctx.saved_tensors
        # one tensor for the three, as the projection that made them takes its gradient
        whole = torch.empty((*x.shape[:-1], 3 * x.shape[-1]), dtype=x.dtype, device=x.device)
        out = whole.unflatten(-1, (3, x.shape[-1])).unbind(-2)
        return c2d.gated_recurrence_backward(grad.contiguous(), x, forget, gate=gate, forget_bias=forget_bias, out=out)


def recurrence(x, forget, gate, forget_bias):
    """gated_recurrence of [batch, tokens, channels] from zero states, with its gradient."""
    return _Recurrence.apply(x, forget, gate, forget_bias)


class TrainedBlock(torch.nn.Module):
    """Projections in 16 or 32 bits, the recurrence between them."""

    def __init__(self, model, inner):
        super().__init__()
        self.into = torch.nn.Linear(model, 3 * inner, bias=False)
        self.out = torch.nn.Linear(inner, model, bias=False)
        self.forget_bias = torch.nn.Parameter(torch.linspace(0.0, 6.0, inner))

    def forward(self, x):
        value, forget, gate = self.into(x).chunk(3, -1)
        return x + self.out(recurrence(value, forget, gate, self.forget_bias))

    def served(self):
        """The weights of the projections in 8 bits, a scale for each output."""
        return c2d.quantize_rows(self.into.weight.detach()), c2d.quantize_rows(self.out.weight.detach())


class GatedRecurrenceBlock:
    def __init__(self, model, batch, inner=None, width=4, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        inner = inner or model
        self.inner = inner

        def weights(out_features, in_features):
            return c2d.quantize_rows(torch.randn(out_features, in_features, generator=g, device=device) / in_features ** 0.5)

        self.into, self.gate, self.out = weights(2 * inner, model), weights(inner, model), weights(model, inner)
        self.conv_w = (torch.randn(inner, width, generator=g, device=device) / width ** 0.5).bfloat16()
        self.forget_bias = torch.rand(inner, generator=g, device=device) * 6
        # the states of `batch` sequences
        self.conv_state = torch.zeros(batch, width - 1, inner, device=device, dtype=torch.bfloat16)
        self.state = torch.zeros(batch, inner, device=device)

    def _project(self, x):
        rows = c2d.quantize_rows(x)
        both = c2d.matmul_q8(rows, self.into)
        return both[:, :self.inner], both[:, self.inner:], c2d.matmul_q8(rows, self.gate)

    def prompt(self, x, lengths, slots, fresh=True):
        """x [tokens, model], the sequences packed; their states end in the rows `slots`."""
        offsets = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).to(x.device)
        packed = {"seq_offsets": offsets, "slots": slots, "fresh": fresh}
        value, forget, gate = self._project(x)
        v = c2d.causal_conv1d(value, self.conv_w, state=self.conv_state, **packed)
        y = c2d.gated_recurrence(v, forget, gate=gate, forget_bias=self.forget_bias, state=self.state, longest=max(lengths),
                                 **packed)
        return c2d.matmul_q8(y, self.out, residual=x)

    def token(self, x, workspace=None):
        """x [batch, model]: the next token of every sequence."""
        value, forget, gate = self._project(x)
        v = c2d.causal_conv1d_step(value, self.conv_w, state=self.conv_state)
        y = c2d.gated_recurrence_step(v, forget, gate=gate, forget_bias=self.forget_bias, state=self.state)
        return c2d.matmul_q8(y, self.out, residual=x, workspace=workspace)

    def record(self, batch, model):
        """(graph, its input, its output, its workspace) of a token step. The warm-up's traces in the states are taken back."""
        x = torch.zeros(batch, model, device=self.state.device, dtype=torch.bfloat16)
        workspace = torch.empty(4 << 20, device=self.state.device, dtype=torch.uint8)
        kept = self.conv_state.clone(), self.state.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.token(x, workspace)
        torch.cuda.current_stream().wait_stream(side)
        self.conv_state.copy_(kept[0])
        self.state.copy_(kept[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = self.token(x, workspace)
        return graph, x, y, workspace


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
    block = GatedRecurrenceBlock(a.model, a.batch)

    # everything as one prompt
    whole = block.prompt(torch.cat(after), [len(x) for x in after], slots).split([len(x) for x in after])
    states = block.conv_state.clone(), block.state.clone()

    # the prompt, then token by token
    prompt = torch.cat([x[:n] for x, n in zip(after, lengths)])
    block.prompt(prompt, lengths, slots)
    graph, x, y, workspace = block.record(a.batch, a.model)
    worst = 0.0
    for t in range(a.tokens):
        x.copy_(torch.stack([s[n + t] for s, n in zip(after, lengths)]))
        graph.replay()
        want = torch.stack([w[n + t] for w, n in zip(whole, lengths)]).float()
        worst = max(worst, float((y.float() - want).norm() / want.norm()))
    drift = [float((s.float() - w.float()).norm() / w.float().norm()) for s, w in zip((block.conv_state, block.state), states)]

    # a training step of the same kind of block, and its weights for serving
    trained = TrainedBlock(a.model, a.model).cuda().bfloat16()
    trained.forget_bias.data = trained.forget_bias.data.float()
    batch = torch.randn(a.batch, min(a.prompt, 512), a.model, generator=g, device="cuda").bfloat16()

    def step():
        trained.zero_grad(set_to_none=True)
        trained(batch).float().square().mean().backward()

    step()
    grads = {name: p.grad for name, p in trained.named_parameters()}
    trained.served()

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
    us_step = timed(step, 10)
    print(f"{a.batch} prompts, {len(prompt)} tokens x {a.model}: {us_prompt:.0f} us ({len(prompt) / us_prompt:.2f} tokens/us)")
    print(f"{a.batch} next tokens: {us_token:.1f} us in a graph, {us_eager:.1f} us call by call")
    print(f"a training step of {batch.shape[0]} x {batch.shape[1]} tokens: {us_step:.0f} us")
    print(f"tokens against one prompt: outputs {worst:.1e}, states {drift[0]:.1e} and {drift[1]:.1e} apart (relative)")
    return worst, drift, grads


if __name__ == "__main__":
    main()
