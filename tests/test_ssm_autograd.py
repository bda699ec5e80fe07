"""The autograd functions of the selective-scan stack, with the operators replaced by
the same formulas in plain torch (no GPU needed): what they keep for the backward pass,
and what they refuse."""
import pytest
import torch

import ssm_ref as ref
from recurrent_cell_unroll_gb300.ssm_block import _Conv, _Scan


class PlainOps:
    """SeqOps' calls by torch's own gradients, in 64 bits."""

    def conv_forward(self, x, weight, bias, lengths, state):
        return ref.conv(x, weight, bias, True, lengths, state)

    def conv_backward(self, dy, x, weight, bias, lengths, state, dstate_n):
        with torch.enable_grad():
            ins = [t.detach().clone().requires_grad_() for t in (x, weight, bias, state)]
            return torch.autograd.grad(self.conv_forward(*ins[:3], lengths, ins[3]), ins, (dy, dstate_n))

    def selscan_forward(self, x, dt, a_log, b, c, d, dt_bias, z, lengths, h0, states):
        return ref.scan(x, dt, a_log, b, c, d, dt_bias, z, lengths, h0)

    def selscan_backward(self, dy, x, dt, a_log, b, c, states, d, dt_bias, z, lengths, dh_n):
        names = ("dx", "ddt", "da_log", "db", "dc", "dd", "ddt_bias", "dz", "dh0")
        with torch.enable_grad():
            ins = [t.detach().clone().requires_grad_() for t in (x, dt, a_log, b, c, d, dt_bias, z, states[0])]
            out = ref.scan(*ins[:8], lengths, ins[8])[:2]
            return dict(zip(names, torch.autograd.grad(out, ins, (dy, dh_n))))


T, B, H, N, W = 4, 2, 3, 2, 3


def leaves(*shapes):
    g = torch.Generator().manual_seed(1)
    return [torch.randn(s, generator=g, dtype=torch.float64).requires_grad_() for s in shapes]


CONV = ((T, B, H), (H, W), (H,), (B, W - 1, H))
SCAN = ((T, B, H), (T, B, H), (H, N), (T, B, N), (T, B, N), (H,), (H,), (T, B, H), (B, H, N))


@pytest.mark.parametrize("lengths", [None, torch.tensor([4, 2])])
def test_gradients(lengths):
    ops = PlainOps()
    assert torch.autograd.gradcheck(lambda *t: _Conv.apply(ops, *t, lengths), leaves(*CONV))
    assert torch.autograd.gradcheck(lambda *t: _Scan.apply(ops, *t, lengths), leaves(*SCAN))


def test_second_derivatives_are_refused():
    ops = PlainOps()
    for fn, shapes in ((_Conv, CONV), (_Scan, SCAN)):
        ins = leaves(*shapes)
        first, = torch.autograd.grad(fn.apply(ops, *ins, None)[0].square().sum(), ins[0], create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            first.square().sum().backward()


def test_lengths_changed_before_the_backward_are_noticed():
    ops = PlainOps()
    for fn, shapes in ((_Conv, CONV), (_Scan, SCAN)):
        lengths = torch.tensor([4, 2])
        y, s = fn.apply(ops, *leaves(*shapes), lengths)
        lengths.copy_(torch.tensor([1, 4]))
        with pytest.raises(RuntimeError, match="inplace"):
            (y.sum() + s.sum()).backward()
