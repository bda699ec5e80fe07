"""A stack of residual blocks around the gated linear recurrence: the sequence
operators together, as a model trains and serves with them.

Each block normalises the residual stream (adding to it what the block before
returned), projects it to the recurrence's input and two gates in one product,
runs the recurrence and projects back:

    u = u + v                      (layernorm_forward's residual)
    n = layer norm(u)
    x | r | i = n W_in             (slices of one product, used where they lie)
    v = recurrence(x, r, i) W_out

For the backward pass a block keeps u and x | r | i, as they are or (act8) as
8-bit checkpoints.  The products are torch.matmul.  ``python -m
recurrent_cell_unroll_gb300.linrec_block`` trains a small stack to repeat its
input some steps later, then serves it token by token.
"""
from __future__ import annotations

import argparse
import math

import torch
from torch.autograd.function import once_differentiable

from . import binding

C = 8.0  # the recurrence's constant


class _Norm(torch.autograd.Function):
    """(y, u) = layer norm of u = x + residual."""

    @staticmethod
    def forward(ctx, ops, act8, x, residual, weight, bias):
        y, u, mean, rstd = ops.layernorm_forward(x, weight, bias, residual=residual)
        ctx.ops, ctx.act8 = ops, act8
        ctx.save_for_backward(*(ops.act8_pack(u) if act8 else (u,)), mean, rstd, weight)
        return y, u

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dsum):
        *u, mean, rstd, weight = ctx.saved_tensors
        du, dw, db = ctx.ops.layernorm_backward(dy, tuple(u) if ctx.act8 else u[0], mean, rstd,
                                                weight, dsum=dsum)
        return None, None, du, du, dw, db


class _Recurrence(torch.autograd.Function):
    """(y, h_n) of the recurrence on z = x | r | i."""

    @staticmethod
    def forward(ctx, ops, act8, z, lam, h0, lengths):
        parts = z.chunk(3, -1)
        y, h_n, states = ops.linrec_forward(*parts, lam, c=C, lengths=lengths, h0=h0, states=True)
        ctx.ops, ctx.act8 = ops, act8
        kept = [t for p in parts for t in ops.act8_pack(p)] if act8 else [z]
        ctx.save_for_backward(lam, states, lengths, *kept)
        return y, h_n

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh_n):
        lam, states, lengths, *kept = ctx.saved_tensors
        parts = [tuple(kept[k:k + 2]) for k in (0, 2, 4)] if ctx.act8 else kept[0].chunk(3, -1)
        dz = torch.empty((*dy.shape[:2], 3 * dy.shape[2]), dtype=dy.dtype, device=dy.device)
        *_, dlam, dh0 = ctx.ops.linrec_backward(dy, *parts, lam, states, c=C, lengths=lengths,
                                                dh_n=dh_n, out=dz)
        return None, None, dz, dlam, dh0, None


class LinRecStack:
    """`layers` blocks of width `dim`, the recurrence `hidden` wide, over [T, B,
    dim] sequences; parameters as torch leaves (float32; products in `dtype`).
    One stream at a time uses a stack: its calls share the workspace of its SeqOps.
    Its gradients can be differentiated once."""

    def __init__(self, layers: int, dim: int, hidden: int, dtype=torch.bfloat16, seed: int = 0,
                 device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def leaf(t):
            return t.to(device).requires_grad_()
        self.ops, self.layers, self.dim, self.hidden = binding.SeqOps(), layers, dim, hidden
        self.dtype, self.device = dtype, device
        self.blocks = []
        for _ in range(layers):
            top = 0.9 + 0.099 * torch.rand(hidden, generator=g)  # a at an open gate
            self.blocks.append({
                "weight": leaf(torch.ones(dim)), "bias": leaf(torch.zeros(dim)),
                "w_in": leaf(torch.randn(dim, 3 * hidden, generator=g) / math.sqrt(dim)),
                "lam": leaf(torch.log(torch.expm1(-torch.log(top) / C))),
                "w_out": leaf(torch.randn(hidden, dim, generator=g) / math.sqrt(hidden))})

    def parameters(self):
        return [t for b in self.blocks for t in b.values()]

    def zero_state(self, batch: int):
        return torch.zeros(self.layers, batch, self.hidden, device=self.device)

    def forward(self, x, state=None, lengths=None, act8=False):
        """Output [T, B, dim] of the whole sequences and the states after them
        [layers, B, hidden].  act8: keep activations in 8 bits."""
        T, B, _ = x.shape
        state = self.zero_state(B) if state is None else state
        u, v, after = x, torch.zeros_like(x), []
        for b, h0 in zip(self.blocks, state):
            n, u = _Norm.apply(self.ops, act8, v, u, b["weight"], b["bias"])
            z = n @ b["w_in"].to(self.dtype)
            y, h_n = _Recurrence.apply(self.ops, act8, z, b["lam"], h0, lengths)
            v = y @ b["w_out"].to(self.dtype)
            after.append(h_n)
        return u + v, torch.stack(after)

    @torch.no_grad()
    def step(self, x, state, slot=None):
        """One token of each request: x [B, dim]; state [layers, slots, hidden]
        is updated in place at the requests' slots (None: row b)."""
        u, v = x, torch.zeros_like(x)
        for b, s in zip(self.blocks, state):
            n, u, _, _ = self.ops.layernorm_forward(v, b["weight"], b["bias"], residual=u)
            z = n @ b["w_in"].to(self.dtype)
            v = self.ops.linrec_step(*z.chunk(3, -1), b["lam"], s, c=C, slot=slot) \
                @ b["w_out"].to(self.dtype)
        return u + v


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--dim", type=int, default=64)
    p.add_argument("--hidden", type=int, default=256)
    p.add_argument("--steps", type=int, default=60, help="training steps")
    p.add_argument("--T", type=int, default=256)
    p.add_argument("--B", type=int, default=16)
    p.add_argument("--delay", type=int, default=4, help="steps after which the input is to be repeated")
    p.add_argument("--act8", action="store_true", help="keep activations in 8 bits")
    a = p.parse_args(argv)
    net = LinRecStack(a.layers, a.dim, a.hidden)
    opt = torch.optim.Adam(net.parameters(), lr=3e-3)
    g = torch.Generator(device="cuda").manual_seed(1)
    losses = []
    for _ in range(a.steps):
        x = torch.randn(a.T, a.B, a.dim, generator=g, device="cuda").to(net.dtype)
        y, _ = net.forward(x, act8=a.act8)
        loss = (y[a.delay:].float() - x[:-a.delay].float()).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    print(f"training: loss {losses[0]:.3f} -> {losses[-1]:.3f} in {a.steps} steps")
    # serving: prefill all but the last tokens, then one by one
    with torch.no_grad():
        whole, _ = net.forward(x)
        out, state = net.forward(x[:-8])
        rest = torch.stack([net.step(t, state) for t in x[-8:]])
    off = float((rest.float() - whole[-8:].float()).abs().max() / whole.float().abs().max())
    print(f"serving: the last 8 tokens one by one, within {off:.1e} of the whole pass")
    assert net.ops.status() == 0
    return losses, off


if __name__ == "__main__":
    main()
