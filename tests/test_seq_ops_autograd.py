"""The autograd functions of the linear-recurrence stack, with the operators replaced
by the same formulas in plain torch (no GPU needed): what they keep for the backward
pass, and what they refuse."""
import pytest
import torch

from recurrent_cell_unroll_gb300.linrec_block import C, _Norm, _Recurrence


class PlainOps:
    """SeqOps' calls by torch's own gradients, in 64 bits."""

    def layernorm_forward(self, x, weight, bias, residual):
        u = x + residual
        mean, rstd = u.mean(-1), (u.var(-1, correction=0) + 1e-5).rsqrt()
        return (u - mean[..., None]) * rstd[..., None] * weight + bias, u, mean, rstd

    def layernorm_backward(self, dy, u, mean, rstd, weight, dsum):
        with torch.enable_grad():
            v, w, b = (t.detach().clone().requires_grad_() for t in (u, weight, torch.zeros_like(weight)))
            y = self.layernorm_forward(v, w, b, torch.zeros_like(v))[0]
            du, dw, db = torch.autograd.grad(y, (v, w, b), dy)
        return du + dsum, dw, db

    def linrec_forward(self, x, r, i, lam, c, lengths, h0, states):
        h, y = h0, []
        for t in range(x.shape[0]):
            a = torch.exp(-c * torch.nn.functional.softplus(lam) * torch.sigmoid(r[t]))
            new = a * h + torch.sqrt(1 - a * a) * torch.sigmoid(i[t]) * x[t]
            on = (t < lengths)[:, None] if lengths is not None else torch.ones(1, 1, dtype=torch.bool)
            h = torch.where(on, new, h)
            y.append(torch.where(on, new, torch.zeros_like(new)))
        return torch.stack(y), h, h0[None]

    def linrec_backward(self, dy, x, r, i, lam, states, c, lengths, dh_n, out):
        with torch.enable_grad():
            ins = [t.detach().clone().requires_grad_() for t in (x, r, i, lam, states[0])]
            y, h, _ = self.linrec_forward(*ins[:4], c, lengths, ins[4], True)
            g = torch.autograd.grad((y, h), ins, (dy, dh_n))
        out.copy_(torch.cat(g[:3], -1))
        return *out.chunk(3, -1), g[3], g[4]


def leaves(*shapes):
    g = torch.Generator().manual_seed(1)
    return [torch.randn(s, generator=g, dtype=torch.float64).requires_grad_() for s in shapes]


def test_gradients():
    ops = PlainOps()
    x, res, w, b = leaves((5, 2, 6), (5, 2, 6), (6,), (6,))
    assert torch.autograd.gradcheck(lambda *t: _Norm.apply(ops, False, *t), (x, res, w, b))
    z, lam, h0 = leaves((5, 2, 9), (3,), (2, 3))
    for lengths in (None, torch.tensor([5, 2])):
        assert torch.autograd.gradcheck(lambda *t: _Recurrence.apply(ops, False, *t, lengths), (z, lam, h0))


def test_second_derivatives_are_refused():
    """The backward passes are kernels without a gradient of their own: asking for one
    raises, where it came without these terms."""
    ops = PlainOps()
    x, res, w, b = leaves((5, 2, 6), (5, 2, 6), (6,), (6,))
    z, lam, h0 = leaves((5, 2, 9), (3,), (2, 3))
    for out, wrt in ((_Norm.apply(ops, False, x, res, w, b)[0], x),
                     (_Recurrence.apply(ops, False, z, lam, h0, None)[0], z)):
        first, = torch.autograd.grad((out * out).sum(), wrt, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (first.square().sum() + wrt.pow(3).sum()).backward()


def test_lengths_changed_before_the_backward_are_noticed():
    """A buffer of lengths that the next batch has been written to: autograd's error for
    saved tensors, not the gradients of other lengths."""
    ops = PlainOps()
    z, lam, h0 = leaves((5, 2, 9), (3,), (2, 3))
    lengths = torch.tensor([5, 2])
    y, h = _Recurrence.apply(ops, False, z, lam, h0, lengths)
    lengths.copy_(torch.tensor([1, 5]))
    with pytest.raises(RuntimeError, match="inplace"):
        (y.sum() + h.sum()).backward()
