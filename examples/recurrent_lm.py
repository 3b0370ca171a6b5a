"""A small recurrent language model on the library's operators: trained on packed
documents, then asked for tokens one at a time.

    python examples/recurrent_lm.py [--steps 400] [--fp32]

A block is layer norm (with the residual added in) -> projection to z_r, z_i, x ->
gated linear recurrence -> projection back; the end is layer norm -> cross entropy
of a linear head that shares the embedding's matrix.  Projections and the optimiser
are torch's.  Training reads whole sequences (glr_fwd, glr_bwd); a prompt is read
by glr_fwd, whose last states go into a pool, and each further token is one
glr_step on that pool.

The documents are made here: a few random tokens, repeated until the document ends,
so that a model with a memory can foresee all but the first period.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import linear_recurrence_scan_diagonal_amd as lrs  # noqa: E402

IGNORED = -1  # a target that counts for nothing


class AddLayerNorm(torch.autograd.Function):
    """(y, s) of s = x + residual, y = layer norm of s."""

    @staticmethod
    def forward(ctx, x, residual, gamma, beta):
        y, s, mean, rstd = lrs.layernorm_fwd(x, gamma, beta, residual=residual, save=True)
        s = x if s is None else s
        ctx.save_for_backward(s, gamma, mean, rstd)
        ctx.has_residual = residual is not None
        return y, s

    @staticmethod
    def backward(ctx, grad_y, grad_s):
        s, gamma, mean, rstd = ctx.saved_tensors
        gx, gg, gb = lrs.layernorm_bwd(s, gamma, mean, rstd, grad_y.contiguous(),
                                       grad_sum=grad_s.contiguous())
        return gx, gx if ctx.has_residual else None, gg, gb


class GatedRecurrence(torch.autograd.Function):
    """h of the gated linear recurrence; z [T,B,3D] holds z_r, z_i and x."""

    @staticmethod
    def forward(ctx, z, bias_r, bias_i, decay, reset):
        parts = z.chunk(3, dim=-1)
        checkpoints = lrs.glr_checkpoints(parts[0])
        h = lrs.glr_fwd(*parts, bias_r, bias_i, decay, reset=reset, checkpoints=checkpoints)
        ctx.save_for_backward(z, bias_r, bias_i, decay, reset, checkpoints)
        return h

    @staticmethod
    def backward(ctx, grad_h):
        z, bias_r, bias_i, decay, reset, checkpoints = ctx.saved_tensors
        grad_z = torch.empty_like(z)
        grads = lrs.glr_bwd(*z.chunk(3, dim=-1), bias_r, bias_i, decay, checkpoints,
                            grad_h.contiguous(), reset=reset, grad_z=grad_z.chunk(3, dim=-1))
        return grad_z, grads[3], grads[4], grads[5], None


class HeadLoss(torch.autograd.Function):
    """Mean cross entropy of x w^T over the targets that are not ignored.  The
    gradient of a mean is known before the loss, so one call gives both and the
    logits are computed once."""

    @staticmethod
    def forward(ctx, x, w, target):
        counted = ((target >= 0) & (target < w.shape[0])).sum().clamp(min=1)
        grad_loss = (1.0 / counted.float()).expand(target.shape[0]).contiguous()
        loss, _, grad_x, grad_w = lrs.linear_ce_fwd_bwd(x, w, target, grad_loss)
        ctx.save_for_backward(grad_x, grad_w)
        return loss.sum() / counted

    @staticmethod
    def backward(ctx, grad):
        grad_x, grad_w = ctx.saved_tensors
        return grad_x * grad.to(grad_x.dtype), grad_w * grad.to(grad_w.dtype), None


class Block(torch.nn.Module):
    def __init__(self, width, device):
        super().__init__()
        self.gamma = torch.nn.Parameter(torch.ones(width, device=device))
        self.beta = torch.nn.Parameter(torch.zeros(width, device=device))
        self.project = torch.nn.Parameter(torch.randn(3 * width, width, device=device) * width**-0.5)
        self.back = torch.nn.Parameter(torch.randn(width, width, device=device) * width**-0.5)
        self.bias_r = torch.nn.Parameter(torch.zeros(width, device=device))
        self.bias_i = torch.nn.Parameter(torch.zeros(width, device=device))
        # memories of a few to some hundred steps
        self.decay = torch.nn.Parameter(torch.linspace(-6.0, -1.0, width, device=device))


class RecurrentLM(torch.nn.Module):
    def __init__(self, vocab, width, blocks, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.dtype = dtype
        self.embedding = torch.nn.Parameter(torch.randn(vocab, width, device=device) * width**-0.5)
        self.blocks = torch.nn.ModuleList(Block(width, device) for _ in range(blocks))
        self.gamma = torch.nn.Parameter(torch.ones(width, device=device))
        self.beta = torch.nn.Parameter(torch.zeros(width, device=device))

    def loss(self, tokens, targets, reset):
        """Mean loss of a packed batch: tokens and targets [T,B] int64, reset [T,B] bool
        (True where a document begins)."""
        w = self.embedding.to(self.dtype)
        x, stream = w[tokens], None
        for b in self.blocks:
            y, stream = AddLayerNorm.apply(x, stream, b.gamma, b.beta)
            z = y @ b.project.to(self.dtype).t()
            h = GatedRecurrence.apply(z, b.bias_r, b.bias_i, b.decay, reset)
            x = h @ b.back.to(self.dtype).t()
        y, _ = AddLayerNorm.apply(x, stream, self.gamma, self.beta)
        return HeadLoss.apply(y.reshape(-1, y.shape[-1]), w, targets.reshape(-1))


class Decoder:
    """Serves a model: one pool of states a block, a row a sequence."""

    def __init__(self, model, slots):
        self.dtype = model.dtype
        self.model = model
        self.w = model.embedding.detach().to(self.dtype)
        self.mats = [(b.project.detach().to(self.dtype).t().contiguous(),
                      b.back.detach().to(self.dtype).t().contiguous()) for b in model.blocks]
        width = self.w.shape[1]
        self.pool = [torch.zeros(slots, width, device=self.w.device) for _ in model.blocks]

    @torch.no_grad()
    def _walk(self, tokens, recurrence):
        x, stream = self.w[tokens], None
        for i, b in enumerate(self.model.blocks):
            project, back = self.mats[i]
            y, s, _, _ = lrs.layernorm_fwd(x, b.gamma, b.beta, residual=stream, out_sum=stream)
            stream = x if s is None else s
            h = recurrence(i, b, (y @ project).chunk(3, dim=-1))
            x = h @ back
        y = lrs.layernorm_fwd(x, self.model.gamma, self.model.beta, residual=stream)[0]
        return y

    def prompt(self, tokens, slots):
        """Reads tokens [T,B] into the pool rows slots [B] (int32, all of them
        rows of the pool).  Returns the logits [B,V] after the last token."""
        rows = slots.long()

        def recurrence(i, b, z):
            h, last = lrs.glr_fwd(*z, b.bias_r, b.bias_i, b.decay, want_h_last=True)
            self.pool[i][rows] = last
            return h
        return self._walk(tokens, recurrence)[-1] @ self.w.t()

    def step(self, tokens, slots):
        """One token [B] for each of the rows slots [B] int32 (outside the pool:
        idle, its logits mean nothing).  Returns the next token's logits [B,V]."""
        def recurrence(i, b, z):
            return lrs.glr_step(*z, b.bias_r, b.bias_i, b.decay, self.pool[i], slots)
        return self._walk(tokens, recurrence) @ self.w.t()


def documents(T, B, vocab, period, length, generator):
    """A packed batch: tokens, targets, reset, [T,B] each.  Documents of up to `length`
    tokens follow each other without a gap; the last token of each, and those of its
    first period, which nothing foretells, have no target."""
    tokens = torch.zeros(T, B, dtype=torch.int64)
    targets = torch.full((T, B), IGNORED, dtype=torch.int64)
    reset = torch.zeros(T, B, dtype=torch.bool)
    for b in range(B):
        t = 0
        while t < T:
            n = min(T - t, int(torch.randint(2 * period, length + 1, (1,), generator=generator)))
            seed = torch.randperm(vocab, generator=generator)[:period]
            doc = seed.repeat(n // period + 1)[:n]
            tokens[t:t + n, b] = doc
            targets[t + period - 1:t + n - 1, b] = doc[period:]
            reset[t, b] = True
            t += n
    return tokens, targets, reset


def train(model, steps, batch, lr=3e-3, report=None):
    """`steps` AdamW steps, batch() giving one batch each; the losses, as floats."""
    opt = torch.optim.AdamW(model.parameters(), lr=lr, weight_decay=0.01)
    losses = []
    for i in range(steps):
        opt.zero_grad(set_to_none=True)
        loss = model.loss(*batch())
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if report and i % report == 0:
            print(f"step {i}: loss {float(losses[-1]):.4f}", flush=True)
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=400)
    ap.add_argument("--fp32", action="store_true", help="fp32 instead of bf16")
    args = ap.parse_args()
    torch.manual_seed(0)
    gen = torch.Generator().manual_seed(1)
    vocab, width, period = 64, 128, 4
    model = RecurrentLM(vocab, width, 2, torch.float32 if args.fp32 else torch.bfloat16)

    def batch():
        return [t.cuda() for t in documents(128, 32, vocab, period, 48, gen)]

    losses = train(model, args.steps, batch, report=20)
    print(f"last loss {losses[-1]:.4f}")

    decoder = Decoder(model, 16)
    prompts = torch.stack([torch.randperm(vocab, generator=gen)[:period].repeat(2)
                           for _ in range(8)], dim=1).cuda()
    slots = torch.arange(8, 16, dtype=torch.int32, device="cuda")
    out = [decoder.prompt(prompts, slots).argmax(-1)]
    for _ in range(2 * period - 1):
        out.append(decoder.step(out[-1], slots).argmax(-1))
    right = (torch.stack(out) == prompts).float().mean()
    print(f"tokens continued as the prompt repeats: {100 * float(right):.0f}%")


if __name__ == "__main__":
    main()
