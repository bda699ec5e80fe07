"""A stack of residual blocks around the selective scan: short convolution, scan and
AdamW together, as a model trains and serves with them.

Each block normalises the residual stream (adding to it what the block before
returned), projects it to the scan's input and gate, filters the input along time,
takes step sizes and weights from it, and projects the scan's output back:

    u = u + v                      (layernorm_forward's residual)
    x | z = layer norm(u) W_in     (slices of one product, used where they lie)
    x = silu(convolution of x along time)
    r | b | c = x W_x,  dt = r W_dt
    v = scan(x, dt, b, c; z) W_out

The products are torch.matmul.  ``python -m recurrent_cell_unroll_gb300.ssm_block``
trains a small stack to repeat its input some steps later, then serves it token by
token.
"""
from __future__ import annotations

import argparse
import math

import torch
from torch.autograd.function import once_differentiable

from . import binding
from .adamw import AdamW
from .linrec_block import _Norm


class _Conv(torch.autograd.Function):
    """(y, state_n) of the short convolution with SiLU."""

    @staticmethod
    def forward(ctx, ops, x, weight, bias, state, lengths):
        y, state_n = ops.conv_forward(x, weight, bias=bias, lengths=lengths, state=state)
        ctx.ops = ops
        ctx.save_for_backward(x, weight, bias, state, lengths)
        return y, state_n

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dstate_n):
        x, weight, bias, state, lengths = ctx.saved_tensors
        dx, dw, db, ds = ctx.ops.conv_backward(dy, x, weight, bias=bias, lengths=lengths, state=state,
                                               dstate_n=dstate_n)
        return None, dx, dw, db, ds, None


class _Scan(torch.autograd.Function):
    """(y, h_n) of the selective scan with its gate."""

    @staticmethod
    def forward(ctx, ops, x, dt, a_log, b, c, d, dt_bias, z, h0, lengths):
        y, h_n, states = ops.selscan_forward(x, dt, a_log, b, c, d=d, dt_bias=dt_bias, z=z,
                                             lengths=lengths, h0=h0, states=True)
        ctx.ops = ops
        ctx.save_for_backward(x, dt, a_log, b, c, d, dt_bias, z, lengths, states)
        return y, h_n

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh_n):
        x, dt, a_log, b, c, d, dt_bias, z, lengths, states = ctx.saved_tensors
        g = ctx.ops.selscan_backward(dy, x, dt, a_log, b, c, states, d=d, dt_bias=dt_bias, z=z,
                                     lengths=lengths, dh_n=dh_n)
        return (None, *(g[k] for k in ("dx", "ddt", "da_log", "db", "dc", "dd", "ddt_bias", "dz",
                                       "dh0")), None)


class SSMStack:
    """`layers` blocks of width `dim`, the scan `hidden` wide with `states` states a
    channel, over [T, B, dim] sequences; parameters as torch leaves (float32; products
    in `dtype`).  One stream at a time uses a stack: its calls share the workspace of
    its SeqOps.  Its gradients can be differentiated once."""

    def __init__(self, layers: int, dim: int, hidden: int, states: int = 16, taps: int = 4,
                 rank: int = 0, dtype=torch.bfloat16, seed: int = 0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def leaf(t):
            return t.to(device).requires_grad_()

        def matrix(rows, cols):
            return leaf(torch.randn(rows, cols, generator=g) / math.sqrt(rows))
        self.ops, self.layers, self.dim, self.hidden = binding.SeqOps(), layers, dim, hidden
        self.states, self.taps, self.rank = states, taps, rank or -(-dim // 16)
        self.dtype, self.device = dtype, device
        self.blocks = []
        for _ in range(layers):
            # step sizes between a thousandth and a tenth at a logit of 0, rates 1 .. states
            step = torch.exp(torch.rand(hidden, generator=g) * math.log(100) + math.log(1e-3))
            rates = torch.log(torch.arange(1.0, states + 1)).repeat(hidden, 1)
            self.blocks.append({
                "weight": leaf(torch.ones(dim)), "bias": leaf(torch.zeros(dim)),
                "w_in": matrix(dim, 2 * hidden),
                "conv": leaf(torch.randn(hidden, taps, generator=g) / math.sqrt(taps)),
                "conv_bias": leaf(torch.zeros(hidden)),
                "w_x": matrix(hidden, self.rank + 2 * states), "w_dt": matrix(self.rank, hidden),
                "dt_bias": leaf(torch.log(torch.expm1(step))), "a_log": leaf(rates),
                "d": leaf(torch.ones(hidden)), "w_out": matrix(hidden, dim)})

    def parameters(self):
        return [t for b in self.blocks for t in b.values()]

    def zero_state(self, batch: int):
        """(windows [layers, batch, taps - 1, hidden], states [layers, batch, hidden, states])."""
        return (torch.zeros(self.layers, batch, self.taps - 1, self.hidden, dtype=self.dtype,
                            device=self.device),
                torch.zeros(self.layers, batch, self.hidden, self.states, device=self.device))

    def _weights(self, b, x, call):
        """What the scan takes beside x: step logits, b and c."""
        r, bw, cw = call(x, b["w_x"]).split([self.rank, self.states, self.states], -1)
        return call(r, b["w_dt"]), bw, cw

    def _product(self, x, w):
        return x @ w.to(self.dtype)

    def forward(self, x, state=None, lengths=None):
        """Output [T, B, dim] of the whole sequences and the state after them."""
        T, B, _ = x.shape
        windows, h0s = self.zero_state(B) if state is None else state
        u, v, after = x, torch.zeros_like(x), ([], [])
        for b, window, h0 in zip(self.blocks, windows, h0s):
            n, u = _Norm.apply(self.ops, False, v, u, b["weight"], b["bias"])
            xs, z = self._product(n, b["w_in"]).chunk(2, -1)
            xs, window_n = _Conv.apply(self.ops, xs, b["conv"], b["conv_bias"], window, lengths)
            dt, bw, cw = self._weights(b, xs, self._product)
            y, h_n = _Scan.apply(self.ops, xs, dt, b["a_log"], bw, cw, b["d"], b["dt_bias"], z, h0, lengths)
            v = self._product(y, b["w_out"])
            after[0].append(window_n)
            after[1].append(h_n)
        return u + v, (torch.stack(after[0]), torch.stack(after[1]))

    @torch.no_grad()
    def step(self, x, state, slot=None):
        """One token of each request: x [B, dim]; state (windows [layers, slots, taps - 1,
        hidden], states [layers, slots, hidden, states]) is updated in place at the
        requests' slots (None: row b)."""
        u, v = x, torch.zeros_like(x)
        for b, window, h in zip(self.blocks, *state):
            n, u, _, _ = self.ops.layernorm_forward(v, b["weight"], b["bias"], residual=u)
            xs, z = self._product(n, b["w_in"]).chunk(2, -1)
            xs = self.ops.conv_step(xs, b["conv"], window, bias=b["conv_bias"], slot=slot)
            dt, bw, cw = self._weights(b, xs, self._product)
            y = self.ops.selscan_step(xs, dt, b["a_log"], bw, cw, h, d=b["d"], dt_bias=b["dt_bias"], z=z,
                                      slot=slot)
            v = self._product(y, b["w_out"])
        return u + v


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--dim", type=int, default=64)
    p.add_argument("--hidden", type=int, default=128)
    p.add_argument("--steps", type=int, default=60, help="training steps")
    p.add_argument("--T", type=int, default=256)
    p.add_argument("--B", type=int, default=16)
    p.add_argument("--delay", type=int, default=3, help="steps after which the input is to be repeated")
    p.add_argument("--opt8", action="store_true", help="keep the optimizer's states in 8 bits")
    a = p.parse_args(argv)
    net = SSMStack(a.layers, a.dim, a.hidden)
    opt = AdamW(net.parameters(), lr=3e-3, weight_decay=0.0, state_bits=8 if a.opt8 else 32, ops=net.ops)
    g = torch.Generator(device="cuda").manual_seed(1)
    losses = []
    for _ in range(a.steps):
        x = torch.randn(a.T, a.B, a.dim, generator=g, device="cuda").to(net.dtype)
        y, _ = net.forward(x)
        loss = (y[a.delay:].float() - x[:-a.delay].float()).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    print(f"training: loss {losses[0]:.3f} -> {losses[-1]:.3f} in {a.steps} steps")
    # serving: prefill all but the last tokens, then one by one
    with torch.no_grad():
        whole, _ = net.forward(x)
        _, state = net.forward(x[:-8])
        rest = torch.stack([net.step(t, state) for t in x[-8:]])
    off = float((rest.float() - whole[-8:].float()).abs().max() / whole.float().abs().max())
    print(f"serving: the last 8 tokens one by one, within {off:.1e} of the whole pass")
    assert net.ops.status() == 0
    return losses, off


if __name__ == "__main__":
    main()
