"""A small language model of linear-attention layers, trained and served with
the layer operators together:

    python examples/linattn_lm.py [--steps 200]

Each layer projects its normed input to q, k, v and a gate, mixes over time by
linear attention with a decay for each head, projects back, and adds the
gated, normed and scaled result to the residual stream, whose norm is the next
layer's input (one fused operator).  Gradients are clipped by their global
norm.  After training the prompt is read in one pass (rows of different
lengths, padded) and continued token by token from the states it left.

The task: a row's first token names one of four permutations, and every other
token is the image of the one before it.  The first token has to be remembered
for the whole row.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import state_space_model_analytic_gb300 as ssd  # noqa: E402

EPS = 1e-5


class LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay, scale):
        ctx.save_for_backward(q, k, v, log_decay)
        ctx.scale = scale
        return ssd.linattn_forward(q, k, v, log_decay, scale=scale, want_state=False)[0]

    @staticmethod
    def backward(ctx, do):
        q, k, v, log_decay = ctx.saved_tensors
        g = ssd.linattn_backward(q, k, v, log_decay, None, do.contiguous(), scale=ctx.scale,
                                 want_dstate0=False)
        return g["dq"], g["dk"], g["dv"], None, None


class BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, residual, y, z, w_post, res_scale, w_pre):
        new, x, stats = ssd.block_norm_forward(residual, y, z, w_post, res_scale, w_pre, EPS)
        ctx.save_for_backward(new, y, z, w_post, res_scale, w_pre, stats)
        return new, x

    @staticmethod
    def backward(ctx, dnew, dx):
        new, y, z, w_post, res_scale, w_pre, stats = ctx.saved_tensors
        g = ssd.block_norm_backward(new, y, z, w_post, res_scale, w_pre, EPS, dx.contiguous(),
                                    dnew.contiguous(), stats)
        return (g["dresidual"], g["dy"], g["dz"], g["dw_post"], g["dres_scale"], g["dw_pre"])


class Model:
    """Weights in fp32, products in bf16, the residual stream in fp32."""

    def __init__(self, vocab=36, width=128, heads=4, dk=32, dv=32, layers=2, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.heads, self.dk, self.dv, self.width = heads, dk, dv, width
        w = lambda *s: (torch.randn(*s, generator=gen) / math.sqrt(s[-1])).cuda()  # noqa: E731
        self.p = {"embed": torch.randn(vocab, width, generator=gen).cuda(), "out": w(vocab, width)}
        cols = heads * (2 * dk + dv) + width  # q, k, v, gate
        for i in range(layers):
            self.p[f"in{i}"] = w(cols, width)
            self.p[f"back{i}"] = w(width, heads * dv)
            self.p[f"post{i}"] = torch.ones(width, device="cuda")
            self.p[f"scale{i}"] = torch.full((width,), 0.5, device="cuda")
            self.p[f"pre{i}"] = torch.ones(width, device="cuda")
        for t in self.p.values():
            t.requires_grad_()
        self.layers = layers
        # heads that remember from a few steps to a few hundred
        self.log_decay = torch.log1p(-torch.exp2(-torch.linspace(2.0, 8.0, heads, device="cuda")))

    def _split(self, x, i):
        """q, k, v and the gate: views of one projection's output."""
        h, dk, dv = self.heads, self.dk, self.dv
        wide = x @ self.p[f"in{i}"].bfloat16().t()
        q, k, v, z = wide.split([h * dk, h * dk, h * dv, self.width], dim=-1)
        return q.unflatten(-1, (h, dk)), k.unflatten(-1, (h, dk)), v.unflatten(-1, (h, dv)), z

    def _start(self, tokens):
        r = self.p["embed"][tokens]
        return r, (r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)).bfloat16()

    def _finish(self, residual, o, z, i, norm):
        y = o.flatten(-2) @ self.p[f"back{i}"].bfloat16().t()
        return norm(residual, y, z, *(self.p[f"{n}{i}"] for n in ("post", "scale", "pre")))

    def logits(self, tokens):
        """Training: [B, T] tokens to [B, T, vocab]."""
        residual, x = self._start(tokens)
        for i in range(self.layers):
            q, k, v, z = self._split(x, i)
            o = LinearAttention.apply(q, k, v, self.log_decay, self.dk ** -0.5)
            residual, x = self._finish(residual, o, z, i, BlockNorm.apply)
        return (x @ self.p["out"].bfloat16().t()).float()

    def _norm(self, *args):
        return ssd.block_norm_forward(*args, EPS, want_stats=False)[:2]

    @torch.no_grad()
    def read(self, tokens, lens):
        """The prompts (row b has lens[b] tokens): last logits and states."""
        residual, x = self._start(tokens)
        states = []
        for i in range(self.layers):
            q, k, v, z = self._split(x, i)
            o, s = ssd.linattn_forward(q, k, v, self.log_decay, scale=self.dk ** -0.5, lens=lens)
            states.append(s)
            residual, x = self._finish(residual, o, z, i, self._norm)
        last = x[torch.arange(len(lens), device="cuda"), lens.long() - 1]
        return (last @ self.p["out"].bfloat16().t()).float(), states

    @torch.no_grad()
    def step(self, tokens, states):
        """One token of every row: next logits; the states move on in place."""
        residual, x = self._start(tokens)
        for i in range(self.layers):
            q, k, v, z = self._split(x, i)
            o, _ = ssd.linattn_step(q, k, v, self.log_decay, states[i], scale=self.dk ** -0.5,
                                    state_out=states[i])
            residual, x = self._finish(residual, o, z, i, self._norm)
        return (x @ self.p["out"].bfloat16().t()).float()


_PERMUTATIONS = torch.stack([torch.randperm(32, generator=torch.Generator().manual_seed(i))
                             for i in range(4)])


def batch(gen, rows, length):
    """[rows, length] tokens: the permutation's name (32 ... 35), then its orbit."""
    which = torch.randint(0, 4, (rows,), generator=gen, device="cuda")
    perm = _PERMUTATIONS.cuda()[which]
    out = [which + 32, torch.randint(0, 32, (rows,), generator=gen, device="cuda")]
    while len(out) < length:
        out.append(perm.gather(1, out[-1][:, None])[:, 0])
    return torch.stack(out, 1)


def train(model, steps, rows=32, length=97, lr=3e-3, max_norm=1.0, seed=1):
    """Adam on the next token, gradients clipped by their global norm; returns
    the losses and the norms."""
    gen = torch.Generator("cuda").manual_seed(seed)
    names = list(model.p)
    m = {n: torch.zeros_like(model.p[n]) for n in names}
    v = {n: torch.zeros_like(model.p[n]) for n in names}
    losses, norms = [], []
    for t in range(1, steps + 1):
        tokens = batch(gen, rows, length)
        logits = model.logits(tokens[:, :-1])
        loss = torch.nn.functional.cross_entropy(logits.flatten(0, 1), tokens[:, 1:].flatten())
        grads = [g.contiguous() for g in torch.autograd.grad(loss, [model.p[n] for n in names])]
        norms.append(ssd.clip_grad_norm(grads, max_norm))
        with torch.no_grad():
            for n, g in zip(names, grads):
                m[n].lerp_(g, 0.1)
                v[n].lerp_(g * g, 0.01)
                step = m[n] / (1 - 0.9 ** t) / ((v[n] / (1 - 0.99 ** t)).sqrt() + 1e-8)
                model.p[n] -= lr * min(1.0, t / 20) * step
        losses.append(loss.detach())
    return [float(x) for x in losses], [float(x) for x in norms]


def generate(model, tokens, lens, count):
    """Greedy continuation of prompts of different lengths: [rows, count]."""
    logits, states = model.read(tokens, lens)
    out = []
    for _ in range(count):
        out.append(logits.argmax(-1))
        logits = model.step(out[-1], states)
    return torch.stack(out, 1)


def main(steps=200, quiet=False):
    model = Model()
    losses, norms = train(model, steps)
    gen = torch.Generator("cuda").manual_seed(99)
    whole = batch(gen, 16, 80)
    lens = torch.randint(30, 61, (16,), generator=gen, device="cuda", dtype=torch.int32)
    got = generate(model, whole[:, :60].contiguous(), lens, 14)
    at = lens.long()[:, None] + torch.arange(14, device="cuda")
    right = float((got == whole.gather(1, at)).float().mean())
    if not quiet:
        print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}, gradient norm {norms[0]:.2f} -> "
              f"{norms[-1]:.2f}, {100 * right:.0f} % of the continuations' tokens right")
    return losses, right


if __name__ == "__main__":
    a = argparse.ArgumentParser()
    a.add_argument("--steps", type=int, default=200)
    main(a.parse_args().steps)
