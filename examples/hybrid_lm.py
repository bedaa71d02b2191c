#!/usr/bin/env python
"""A small hybrid language model on libgla: pre-norm blocks that alternate GLA layers (matrix state) with gated linear
recurrences (vector state), trained for a few steps and then served token by token.

    python examples/hybrid_lm.py                 # train on a synthetic task, then generate
    python examples/hybrid_lm.py --steps 50 --dtype fp32

The layer operators come from the binding: ``norm_fwd`` / ``norm_bwd`` around the residual stream (kept in fp32),
``gla_fwd`` / ``gla_bwd`` and ``scan_fwd`` / ``scan_bwd`` over sequences, ``gla_step`` and ``scan_step`` for single
tokens on state pools, and ``norm_quant_fwd`` where decoding takes its activations in 8 bits.  The projections are
torch matrix products.  Synthetic data: token t + 1 is a fixed permutation of token t, one in ten replaced at random.
"""
import argparse
import os
import sys
import time

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from chunkwise_gated_linear_chunked_gb300 import binding  # noqa: E402

VOCAB, HEADS, HEAD_DIM, LAYERS = 32, 2, 64, 4
WIDTH = HEADS * HEAD_DIM


class Norm(torch.autograd.Function):
    """(y, s): s = x + res on the fp32 residual stream, y its norm in x's type."""

    @staticmethod
    def forward(ctx, x, res, w):
        y, s, rstd = binding.norm_fwd(x, residual=res, weight=w)
        ctx.save_for_backward(s, rstd, w)
        return y, s

    @staticmethod
    def backward(ctx, dy, ds):
        s, rstd, w = ctx.saved_tensors
        return binding.norm_bwd(s, rstd, dy.contiguous(), weight=w, ds=ds.contiguous())


class Gla(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g):
        ctx.save_for_backward(q, k, v, g)
        return binding.gla_fwd(q, k, v, g)[0]

    @staticmethod
    def backward(ctx, do):
        q, k, v, g = ctx.saved_tensors
        grads = binding.gla_bwd(q, k, v, g, do.to(q.dtype).contiguous(), want_dh0=False)[:4]
        return tuple(d.to(q.dtype) for d in grads)


class Scan(torch.autograd.Function):
    """The recurrence on the two halves (input, gate) of a projection's output, as they lie there."""

    @staticmethod
    def forward(ctx, xg):
        x, g = xg[..., :WIDTH], xg[..., WIDTH:]
        h, _ = binding.scan_fwd(x, g, out_dtype=x.dtype)
        ctx.save_for_backward(xg, h)
        return h

    @staticmethod
    def backward(ctx, dh):
        xg, h = ctx.saved_tensors
        grad = torch.empty_like(xg)
        binding.scan_bwd(xg[..., WIDTH:], h, dh.contiguous(), dx=grad[..., :WIDTH], dg=grad[..., WIDTH:], want_dh0=False)
        return grad


def log_gate(logits, sharpness):
    """Log-decay below zero from a gate's logits."""
    return F.logsigmoid(logits.float()) / sharpness


class Model:
    def __init__(self, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device=device, generator=gen)  # noqa: E731
        self.dtype, self.device = dtype, device
        self.p = {"embed": rand(VOCAB, WIDTH), "norm_out": torch.ones(WIDTH, device=device),
                  "logits": rand(VOCAB, WIDTH) / WIDTH ** 0.5}
        for i in range(LAYERS):
            wide = 4 if self.is_gla(i) else 2
            self.p[f"norm{i}"] = torch.ones(WIDTH, device=device)
            self.p[f"in{i}"] = rand(wide * WIDTH, WIDTH) / WIDTH ** 0.5
            self.p[f"out{i}"] = 0.5 * rand(WIDTH, WIDTH) / WIDTH ** 0.5

    @staticmethod
    def is_gla(i):
        return i % 2 == 0

    def weight(self, name):
        return self.p[name].to(self.dtype)

    def split(self, i, z):
        """A layer's operands from its projection's output z [..., wide * WIDTH]."""
        if self.is_gla(i):
            q, k, v, gate = (t.reshape(*t.shape[:-1], HEADS, HEAD_DIM) for t in z.chunk(4, -1))
            return q.contiguous(), k.contiguous(), v.contiguous(), log_gate(gate, 16).to(self.dtype)
        x, gate = z.chunk(2, -1)
        return torch.cat([x, log_gate(gate, 4).to(self.dtype)], -1)

    def forward(self, tokens, states=None):
        """Logits [B, T, VOCAB].  With ``states`` (a list) each layer's final state is appended to it (no gradients)."""
        stream = self.p["embed"][tokens]                              # fp32 residual stream
        x = torch.zeros_like(stream, dtype=self.dtype)
        for i in range(LAYERS):
            y, stream = Norm.apply(x, stream, self.p[f"norm{i}"])
            operands = self.split(i, y @ self.weight(f"in{i}").T)
            if states is not None:
                o, state = binding.gla_fwd(*operands) if self.is_gla(i) else \
                    binding.scan_fwd(operands[..., :WIDTH], operands[..., WIDTH:], out_dtype=self.dtype)
                states.append(state)
            else:
                o = Gla.apply(*operands) if self.is_gla(i) else Scan.apply(operands)
            x = o.reshape(stream.shape).to(self.dtype) @ self.weight(f"out{i}").T
        y, _ = Norm.apply(x, stream, self.p["norm_out"])
        return (y @ self.weight("logits").T).float()


def batch(n, length, seed, device="cuda"):
    gen = torch.Generator().manual_seed(seed)
    follow = torch.randperm(VOCAB, generator=torch.Generator().manual_seed(7))
    tokens = torch.randint(VOCAB, (n, length + 1), generator=gen)
    keep = torch.rand(n, length + 1, generator=gen) < 0.9
    for t in range(1, length + 1):
        tokens[:, t] = torch.where(keep[:, t], follow[tokens[:, t - 1]], tokens[:, t])
    return tokens.to(device)


def train(model, steps, n=8, length=200, rate=3e-3):
    """Adam on the next-token loss; returns the losses."""
    for w in model.p.values():
        w.requires_grad_(True)
    opt = torch.optim.Adam(model.p.values(), lr=rate)
    losses = []
    for step in range(steps):
        tokens = batch(n, length, step, model.device)
        loss = F.cross_entropy(model.forward(tokens[:, :-1]).reshape(-1, VOCAB), tokens[:, 1:].reshape(-1))
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    for w in model.p.values():
        w.requires_grad_(False)
    return torch.stack(losses).tolist()


class Server:
    """Decodes up to ``slots`` sequences, one token each a call; their states live in pools, updated in place."""

    def __init__(self, model, slots, eight_bit=False):
        self.m, self.eight_bit = model, eight_bit
        shape = lambda i: (HEADS, HEAD_DIM, HEAD_DIM) if model.is_gla(i) else (WIDTH,)  # noqa: E731
        self.pools = [torch.zeros(slots, *shape(i), device=model.device) for i in range(LAYERS)]
        self.w = {n: model.weight(n).T.contiguous() for n in model.p if n.startswith(("in", "out", "logits"))}

    def prefill(self, tokens, slots):
        """Runs whole prompts [B, T] and leaves their states in the pools; returns the last logits [B, VOCAB]."""
        states = []
        logits = self.m.forward(tokens, states)
        for pool, state in zip(self.pools, states):
            pool[slots.long()] = state
        return logits[:, -1]

    def project(self, x, stream, norm, weight):
        """(norm of x + stream) times a weight, and the new stream; the norm's output in 8 bits if asked."""
        if not self.eight_bit:
            y, stream, _ = binding.norm_fwd(x, residual=stream, weight=self.m.p[norm])
            return y @ self.w[weight], stream
        q, scales, stream, _ = binding.norm_quant_fwd(x, residual=stream, weight=self.m.p[norm])
        return ((q.to(self.m.dtype) @ self.w[weight]) * scales).to(self.m.dtype), stream

    def step(self, tokens, slots):
        """The next logits [B, VOCAB] after one more token [B] of each sequence."""
        stream = self.m.p["embed"][tokens]
        x = torch.zeros_like(stream, dtype=self.m.dtype)
        for i, pool in enumerate(self.pools):
            z, stream = self.project(x, stream, f"norm{i}", f"in{i}")
            operands = self.m.split(i, z)
            if self.m.is_gla(i):
                o = binding.gla_step(*operands, pool, slots=slots).to(self.m.dtype)
            else:
                o = binding.scan_step(operands[:, :WIDTH], operands[:, WIDTH:], pool, slots=slots, out_dtype=self.m.dtype)
            x = o.reshape(x.shape) @ self.w[f"out{i}"]
        return self.project(x, stream, "norm_out", "logits")[0].float()


def generate(server, prompt, slots, count):
    """``count`` greedy tokens after each prompt, the token loop's body captured once in a CUDA graph."""
    tokens = server.prefill(prompt, slots).argmax(-1)
    kept = [pool.clone() for pool in server.pools]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        server.step(tokens, slots)   # before the capture: libraries set themselves up
    torch.cuda.current_stream().wait_stream(side)
    for pool, was in zip(server.pools, kept):
        pool.copy_(was)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens_next = server.step(tokens, slots).argmax(-1)
    out = [tokens.clone()]
    for _ in range(count - 1):
        graph.replay()
        tokens.copy_(tokens_next)
        out.append(tokens.clone())
    return torch.stack(out, 1)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--dtype", choices=["bf16", "fp32"], default="bf16")
    ap.add_argument("--eight-bit", action="store_true", help="decode with activations in 8 bits")
    a = ap.parse_args()
    model = Model(torch.bfloat16 if a.dtype == "bf16" else torch.float32)
    losses = train(model, a.steps)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {a.steps} steps")
    prompts = batch(16, 99, 1000)
    slots = torch.randperm(32, generator=torch.Generator().manual_seed(1))[:16].to("cuda", torch.int32)
    start = time.perf_counter()
    out = generate(Server(model, 32, a.eight_bit), prompts, slots, 64)
    follow = torch.randperm(VOCAB, generator=torch.Generator().manual_seed(7)).cuda()
    right = (out[:, 1:] == follow[out[:, :-1]]).float().mean()
    if binding.layer_status() != binding.GLA_OK:
        raise SystemExit("a kernel reported bad slots or offsets")
    print(f"64 tokens for 16 sequences in {time.perf_counter() - start:.2f} s; {100 * right:.0f} % follow the rule")


if __name__ == "__main__":
    main()
